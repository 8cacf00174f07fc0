"""A stack of layers with its residual paths, loss and clipping against the same in 64 bits, as a training and a serving program run it.

The layers pick every expert (k = E), so no rounding changes the routing and the
stack is a smooth function.  Tolerances are those of the layer: 2e-2 of the
largest value for bf16, 1e-4 for float32.
"""
import math

import numpy as np
import pytest
import torch

import routing_permute_grouped_router_gb300 as pkg
from _util import TOL, assert_close, check_no_device_error
from routing_permute_grouped_router_gb300 import layer as L

pytestmark = pytest.mark.gpu
SHAPES = {"f32": (33, 64, 36, 3, 101), "bf16": (200, 256, 256, 2, 1000)}


@pytest.fixture(scope="module", autouse=True)
def built():
    from routing_permute_grouped_router_gb300 import build

    build.build()
    pkg.lib()
    torch.cuda.set_device(0)
    pkg.moe_get_device_error(clear=True)


def make(kind, n=2, training=True, T=None, post=True, gate=True, seed=3):
    t, (T0, d, f, E, V) = (torch.float32 if kind == "f32" else torch.bfloat16), SHAPES[kind]
    T = T0 if T is None else T
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s, scale=1.0, to=t: (torch.randn(*s, generator=g, device="cuda") * scale).to(to)  # noqa: E731
    cfg = pkg.config(T, d, f, E, E, 0.0, -1, pkg.MOE_F32 if kind == "f32" else pkg.MOE_BF16)
    f32 = torch.float32
    layers = [L.MoELayer(cfg, rand(d, E, scale=d ** -0.5, to=f32), None, rand(E, d, f, scale=d ** -0.5),
                         rand(E, d, f, scale=d ** -0.5), rand(E, f, d, scale=f ** -0.5), training) for _ in range(n)]
    vec = lambda: 1 + rand(d, scale=0.2, to=f32)  # noqa: E731
    stack = L.MoEStack(layers, [vec() for _ in range(n + 1)], [vec() for _ in range(n)] if post else None,
                       [vec() for _ in range(n)] if gate else None, rand(V, d, scale=d ** -0.5), 0.9, 0.7)
    x = rand(T, d)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    labels[::5] = -100
    return stack, x, labels


def reference(stack, x, labels, dloss=None):
    """Loss of each token, and the gradients of its mean or of sum(dloss loss), by autograd in 64 bits; moe_clip_grads' norm of them."""
    leaf = lambda v: v.detach().double().requires_grad_(True)  # noqa: E731
    xs, head = leaf(x), leaf(stack.head)
    gam = [leaf(v) for v in stack.gammas]
    post = [None if v is None else leaf(v) for v in stack.posts]
    gate = [None if v is None else leaf(v) for v in stack.gates]
    w = [{n: leaf(l.weights[n]) for n in ("W_r", "W1", "W3", "W2")} for l in stack.layers]

    def norm(v, g):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + stack.eps) * g

    s, h = xs, norm(xs, gam[0])
    for i, p in enumerate(w):
        gates = torch.softmax(h @ p["W_r"], 1)
        a, b = torch.einsum("td,edf->etf", h, p["W1"]), torch.einsum("td,edf->etf", h, p["W3"])
        y = torch.einsum("te,etf,efd->td", gates, a * torch.sigmoid(a) * b, p["W2"])
        u = y if post[i] is None else norm(y, post[i])
        s = stack.residual_scale * s + stack.branch_scale * (u if gate[i] is None else gate[i] * u)
        h = norm(s, gam[i + 1])
    z = h @ head.t()
    valid = labels >= 0
    per = torch.where(valid, torch.logsumexp(z, 1) - z.gather(1, labels.long().clamp(min=0)[:, None])[:, 0], 0.0)
    (per.sum() / valid.sum() if dloss is None else (per * dloss.double()).sum()).backward()
    grads = [p[n].grad for p in w for n in ("W_r", "W1", "W3", "W2")]
    grads += [v.grad for group in (gam, post, gate, [head]) for v in group if v is not None]
    return per.detach(), h.detach(), xs.grad, grads


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("post,gate", [(True, True), (False, False), (True, False)])
def test_stack_step(kind, post, gate):
    stack, x, labels = make(kind, post=post, gate=gate)
    per, h, dx, grads = reference(stack, x, labels)
    total = stack.forward_loss(x, labels)
    got_dx = stack.backward(x, labels, False)
    torch.cuda.synchronize()
    check_no_device_error()
    tol = TOL[kind]
    assert_close("h", stack.h[-1], h.cpu(), tol)
    assert_close("loss", stack.loss, per.cpu(), tol)
    assert int(total[1]) == int((labels >= 0).sum()) and abs(float(total[0]) - float(per.sum())) <= tol * float(per.sum())
    assert_close("dx", got_dx, dx.cpu(), tol)
    got = stack.gradients()
    assert len(got) == len(grads)
    for i, (a, b) in enumerate(zip(got, grads)):
        assert_close(f"gradient {i}", a, b.cpu(), tol)
    norm = math.sqrt(sum(float(b.square().sum()) for b in grads))
    before = [a.clone() for a in got]
    assert abs(float(stack.clip(norm / 4)) - norm) <= tol * norm
    scale = norm / 4 / math.sqrt(sum(float(a.double().square().sum()) for a in before))
    for a, b in zip(stack.gradients(), before):
        assert (a.double() - b.double() * scale).abs().max() <= 2e-6 * b.abs().max()


def test_stack_two_micro_batches_add_up():
    stack, x, labels = make("f32")
    _, x2, labels2 = make("f32", seed=5)
    w = torch.rand(x.shape[0], device="cuda")
    a, b = reference(stack, x, labels, w)[3], reference(stack, x2, labels2, w)[3]
    for xs, ls, acc in ((x, labels, False), (x2, labels2, True)):
        stack.forward_loss(xs, ls)
        stack.backward(xs, ls, acc, w)
    for i, (g, u, v) in enumerate(zip(stack.gradients(), a, b)):
        assert_close(f"gradient {i}", g, (u + v).cpu(), TOL["f32"])
    check_no_device_error()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_stack_step_captured(kind):
    """Forward, loss, backward and clipping in one graph, on a stream of its own."""
    stack, x, labels = make(kind)

    def step():
        stack.forward_loss(x, labels)
        stack.backward(x, labels, False)
        stack.clip(0.5)

    step()
    first = [v.clone() for v in (stack.total, stack.dx, stack.norm, *stack.gradients())]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        for v in (stack.total, stack.dx, stack.norm, *stack.gradients()):
            v.fill_(float("nan"))
        g.replay()
        g.replay()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (stack.total, stack.dx, stack.norm, *stack.gradients())))
    check_no_device_error()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_stack_decode(kind):
    stack, x, labels = make(kind, training=False)
    full = stack.forward(x).double()
    for T in (1, 7, 33):
        out = stack.decode(x[:T].contiguous())
        assert_close("decode", out, full[:T].cpu(), TOL[kind])
        # and the tokens' scores over the vocabulary
        ws = pkg.vocab_loss_workspace(T, x.shape[1], stack.head.shape[0], x.dtype, False)
        loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        pkg.moe_vocab_loss_fwd(out, stack.head, labels[:T].contiguous(), loss, lse, ws)
        z = out.double() @ stack.head.double().t()
        exp = torch.where(labels[:T] >= 0, torch.logsumexp(z, 1) - z.gather(1, labels[:T].long().clamp(min=0)[:, None])[:, 0], 0.0)
        assert_close("score", loss, exp.cpu(), 1e-5)
    check_no_device_error()


@pytest.mark.parametrize("n", [1, 2])
def test_stack_decode_of_its_own_result(n):
    """The buffer that a call returns is the next call's input; and calls on two streams keep apart."""
    stack, x, _ = make("f32", n=n, training=False)
    first = stack.decode(x[:8].contiguous()).clone()
    again = stack.decode(first.clone()).clone()
    out = stack.decode(x[:8].contiguous())
    assert torch.equal(stack.decode(out), again)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = stack.decode(x[:8].contiguous(), s)
    here = stack.decode(first)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(other, first) and torch.equal(here, again) and other.data_ptr() != here.data_ptr()
    assert stack.decode(x[:0]).shape == (0, 64)
    check_no_device_error()


def test_stack_of_no_tokens():
    stack, x, labels = make("f32", T=0)
    assert stack.forward_loss(x, labels).tolist() == [0.0, 0.0]
    assert stack.backward(x, labels, False).shape == (0, 64)
    assert float(stack.clip(1.0)) == 0.0 and not any(g.any() for g in stack.gradients())
    check_no_device_error()


def test_stack_refuses():
    stack, x, labels = make("f32", training=False)
    with pytest.raises(RuntimeError, match="training buffers"):
        stack.backward(x, labels, False)
    with pytest.raises(RuntimeError, match="training buffers"):
        stack.clip(1.0)
    with pytest.raises(ValueError, match="n \\+ 1 norms"):
        L.MoEStack(stack.layers, stack.gammas[:2])
    with pytest.raises(ValueError, match="same tokens"):
        L.MoEStack([stack.layers[0], make("f32", T=5)[0].layers[0]], stack.gammas)
    with pytest.raises(ValueError, match="twice"):
        L.MoEStack([stack.layers[0], stack.layers[0]], stack.gammas)
    for bad, err in ((x.half(), TypeError), (x[:65].repeat(3, 1), pkg.MoeError)):
        with pytest.raises(err):
            stack.decode(bad)
    bare = L.MoEStack(stack.layers, stack.gammas)
    with pytest.raises(RuntimeError, match="without a head"):
        bare.forward_loss(x, labels)
    assert np.isfinite(bare.forward(x).cpu().numpy()).all()
