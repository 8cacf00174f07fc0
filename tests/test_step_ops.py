"""Operators that join blocks to a training step, without a GPU: refusals, workspaces, the 64-bit forms themselves."""
import ctypes

import pytest
import torch

import _step_ref as ref
import routing_permute_grouped_router_gb300 as pkg
from routing_permute_grouped_router_gb300 import build as B

P, Q, R, S = 0x1000, 0x2000, 0x3000, 0x4000  # never followed: each call here is refused before a launch


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pkg.lib()


@pytest.fixture(autouse=True)
def no_launch(lib):
    n = lib.moe_launch_count()
    yield
    assert lib.moe_launch_count() == n


def status(rc):
    return pkg.STATUS[rc]


def join(**kw):
    a = dict(rows=4, d=64, dtype=pkg.MOE_BF16, gamma_post=P, gamma_next=P, gate=None, row_gate=None, residual_scale=1.0,
             branch_scale=1.0, eps=1e-6)
    a.update(kw)
    return pkg.MoeResidualNorm(*[a[n] for n, _ in pkg.MoeResidualNorm._fields_])


@pytest.mark.parametrize("kw,err", [
    (dict(dtype=7), "MOE_ERR_DTYPE"), (dict(rows=-1), "MOE_ERR_SHAPE"), (dict(d=0), "MOE_ERR_SHAPE"),
    (dict(d=65537), "MOE_ERR_SHAPE"), (dict(rows=1 << 40, d=2), "MOE_ERR_SHAPE"),
    (dict(eps=-1.0), "MOE_ERR_INVALID_ARG"), (dict(eps=float("nan")), "MOE_ERR_INVALID_ARG"),
    (dict(residual_scale=float("inf")), "MOE_ERR_INVALID_ARG"), (dict(branch_scale=float("nan")), "MOE_ERR_INVALID_ARG"),
    (dict(gamma_post=P + 2), "MOE_ERR_ALIGNMENT"), (dict(gate=P + 1), "MOE_ERR_ALIGNMENT"),
])
def test_join_refuses_configurations(lib, kw, err):
    p = join(**kw)
    assert status(lib.moe_residual_norm_fwd(ctypes.byref(p), P, P, Q, R, None, None, None)) == err
    assert status(lib.moe_residual_norm_bwd(ctypes.byref(p), P, P, P, P, P, P, Q, R, None, 0, P, 1 << 40, None)) == err


@pytest.mark.parametrize("kw,x,y,out,h,ry,ro,err", [
    ({}, None, P, Q, R, None, None, "MOE_ERR_INVALID_ARG"),
    ({}, P + 8, P, Q, R, None, None, "MOE_ERR_ALIGNMENT"),
    ({}, P, P + 4, Q, R, None, None, "MOE_ERR_ALIGNMENT"),
    ({}, P, None, Q, R, None, None, "MOE_ERR_INVALID_ARG"),                                   # a norm of no branch
    (dict(gamma_post=None, gate=P), P, None, Q, R, None, None, "MOE_ERR_INVALID_ARG"),        # a gate of no branch
    ({}, P, P, Q, None, None, None, "MOE_ERR_INVALID_ARG"),                                   # no place for h
    (dict(gamma_next=None), P, P, Q, R, None, None, "MOE_ERR_INVALID_ARG"),                   # h without its weight
    (dict(gamma_next=None), P, P, None, None, None, None, "MOE_ERR_INVALID_ARG"),             # nothing to write
    (dict(gamma_next=None), P, P, Q, None, None, S, "MOE_ERR_INVALID_ARG"),
    (dict(gamma_post=None), P, P, Q, R, S, None, "MOE_ERR_INVALID_ARG"),
    ({}, P, P, Q, Q, None, None, "MOE_ERR_INVALID_ARG"),                                      # out is h
    ({}, P, P, Q, R, S + 2, None, "MOE_ERR_ALIGNMENT"),
])
def test_join_fwd_refuses(lib, kw, x, y, out, h, ry, ro, err):
    assert status(lib.moe_residual_norm_fwd(ctypes.byref(join(**kw)), x, y, out, h, ry, ro, None)) == err


def test_join_bwd_refuses(lib):
    def call(kw={}, out=P, y=P, dh=P, dout=P, ry=P, ro=P, dx=Q, dy=R, g=None, acc=0, ws=P, n=1 << 40):
        gr = None if g is None else ctypes.byref(pkg.MoeResidualNormGrads(**g))
        return status(lib.moe_residual_norm_bwd(ctypes.byref(join(**kw)), out, y, dh, dout, ry, ro, dx, dy, gr, acc, ws, n, None))

    bad = "MOE_ERR_INVALID_ARG"
    assert call(acc=2) == bad
    assert call(out=None) == bad and call(y=None) == bad and call(dh=None) == bad and call(dy=None) == bad
    assert call(ry=None) == bad and call(ro=None) == bad and call(dx=Q, dy=Q) == bad
    assert call(dict(gamma_next=None)) == bad                                  # dh without a norm
    assert call(dict(gamma_next=None), dh=None, dout=None) == bad
    for name, kw in (("dgamma_post", dict(gamma_post=None)), ("dgamma_next", dict(gamma_next=None)), ("dgate", {}), ("drow_gate", {})):
        assert call(kw, g={name: P}, dh=None if "gamma_next" in kw else P) == bad
    assert call(dx=Q + 4) == "MOE_ERR_ALIGNMENT" and call(g=dict(dgamma_post=P + 1)) == "MOE_ERR_ALIGNMENT"
    assert call(ws=None) == "MOE_ERR_WORKSPACE" and call(n=16) == "MOE_ERR_WORKSPACE"
    assert status(lib.moe_residual_norm_fwd(None, P, P, Q, R, None, None, None)) == bad


def test_join_workspace(lib):
    with pytest.raises(pkg.MoeError, match="SHAPE"):
        pkg.moe_residual_norm_workspace_size(-1, 8)
    sizes = [pkg.moe_residual_norm_workspace_size(r, d) for r, d in ((0, 8), (1, 1), (4099, 1021), (32768, 4096), (7, 65536))]
    assert all(s > 0 for s in sizes)


def grads(*entries):
    return (pkg.MoeGrad * len(entries))(*[pkg.MoeGrad(*e) for e in entries])


F, H = pkg.MOE_F32, pkg.MOE_BF16


@pytest.mark.parametrize("entries,norm,most,ws,err", [
    ([(P, None, 4, F)], None, 1.0, 1 << 30, "MOE_ERR_INVALID_ARG"),
    ([(P, None, 4, F)], S + 2, 1.0, 1 << 30, "MOE_ERR_ALIGNMENT"),
    ([(P, None, 4, F)], S, 0.0, 1 << 30, "MOE_ERR_INVALID_ARG"),
    ([(P, None, 4, F)], S, -1.0, 1 << 30, "MOE_ERR_INVALID_ARG"),
    ([(P, None, 4, F)], S, float("nan"), 1 << 30, "MOE_ERR_INVALID_ARG"),
    ([(P, None, 4, F)], S, 1.0, 100, "MOE_ERR_WORKSPACE"),
    ([(P, None, 4, 5)], S, 1.0, 1 << 30, "MOE_ERR_DTYPE"),
    ([(P, None, -1, F)], S, 1.0, 1 << 30, "MOE_ERR_SHAPE"),
    ([(P, None, (1 << 40) + 1, F)], S, 1.0, 1 << 30, "MOE_ERR_SHAPE"),
    ([(None, None, 4, F)], S, 1.0, 1 << 30, "MOE_ERR_INVALID_ARG"),
    ([(P + 2, None, 4, F)], S, 1.0, 1 << 30, "MOE_ERR_ALIGNMENT"),
    ([(P + 1, None, 4, H)], S, 1.0, 1 << 30, "MOE_ERR_ALIGNMENT"),
    ([(P, Q + 2, 4, F)], S, 1.0, 1 << 30, "MOE_ERR_ALIGNMENT"),
    ([(P, P, 4, F), (P, P, 4, F)], S, 1.0, 1 << 30, "MOE_ERR_INVALID_ARG"),          # the same tensor twice
    ([(P, Q, 4, F), (R, Q + 12, 4, F)], S, 1.0, 1 << 30, "MOE_ERR_INVALID_ARG"),     # destinations overlap
    ([(P, P + 4, 4, F)], S, 1.0, 1 << 30, "MOE_ERR_INVALID_ARG"),                    # overlaps its own source
    ([(P, None, 8, F), (Q, P + 16, 4, F)], S, 1.0, 1 << 30, "MOE_ERR_INVALID_ARG"),  # overlaps another source
    ([(P, Q, 8, F)] + [(0x100000 + 64 * i, None, 16, F) for i in range(60)] + [(R, 0x100000 + 64 * 59 + 60, 1, F)], S,
     1.0, 1 << 30, "MOE_ERR_INVALID_ARG"),
])
def test_clip_refuses(lib, entries, norm, most, ws, err):
    assert status(lib.moe_clip_grads(grads(*entries), len(entries), most, norm, P, ws, None)) == err


def test_clip_counts(lib):
    for n in (-1, pkg.MOE_CLIP_MAX_TENSORS + 1):
        assert status(lib.moe_clip_grads(None, n, 1.0, S, P, 1 << 30, None)) == "MOE_ERR_SHAPE"
        with pytest.raises(pkg.MoeError, match="SHAPE"):
            pkg.moe_clip_workspace_size(n)
    assert status(lib.moe_clip_grads(None, 3, 1.0, S, P, 1 << 30, None)) == "MOE_ERR_INVALID_ARG"
    assert pkg.moe_clip_workspace_size(0) > 0
    assert pkg.moe_clip_workspace_size(pkg.MOE_CLIP_MAX_TENSORS) >= pkg.moe_clip_workspace_size(100)


def test_grad_list_checks():
    t = torch.zeros(4)
    with pytest.raises(TypeError):
        pkg.grad_list([t.half()])
    with pytest.raises(ValueError, match="CUDA"):
        pkg.grad_list([t])
    with pytest.raises(ValueError, match="destinations"):
        pkg.grad_list([t], [])


def loss_fwd(lib, T=4, d=64, V=100, dtype=H, x=P, W=Q, labels=R, loss=S, lse=S, total=None, ws=P, n=1 << 44):
    return status(lib.moe_vocab_loss_fwd(T, d, V, dtype, x, W, labels, loss, lse, total, ws, n, None))


def loss_bwd(lib, T=4, d=64, V=100, dtype=H, dw=F, x=P, W=Q, labels=R, lse=S, dloss=None, dx=Q, dW=R, acc=0, ws=P, n=1 << 44):
    return status(lib.moe_vocab_loss_bwd(T, d, V, dtype, dw, x, W, labels, lse, dloss, dx, dW, acc, ws, n, None))


@pytest.mark.parametrize("kw,err", [
    (dict(dtype=3), "MOE_ERR_DTYPE"), (dict(T=-1), "MOE_ERR_SHAPE"), (dict(T=(1 << 24) + 1), "MOE_ERR_SHAPE"),
    (dict(V=0), "MOE_ERR_SHAPE"), (dict(V=(1 << 24) + 1), "MOE_ERR_SHAPE"), (dict(d=0), "MOE_ERR_SHAPE"),
    (dict(d=68), "MOE_ERR_SHAPE"), (dict(d=66, dtype=F), "MOE_ERR_SHAPE"), (dict(d=65544), "MOE_ERR_SHAPE"),
    (dict(x=None), "MOE_ERR_INVALID_ARG"), (dict(W=None), "MOE_ERR_INVALID_ARG"), (dict(labels=None), "MOE_ERR_INVALID_ARG"),
    (dict(lse=None), "MOE_ERR_INVALID_ARG"), (dict(x=P + 8), "MOE_ERR_ALIGNMENT"), (dict(W=Q + 2), "MOE_ERR_ALIGNMENT"),
    (dict(labels=R + 2), "MOE_ERR_ALIGNMENT"), (dict(ws=None), "MOE_ERR_WORKSPACE"), (dict(n=1000), "MOE_ERR_WORKSPACE"),
])
def test_loss_refuses(lib, kw, err):
    assert loss_fwd(lib, **kw) == err
    assert loss_bwd(lib, **kw) == err


def test_loss_refuses_one_way(lib):
    assert loss_fwd(lib, loss=None) == "MOE_ERR_INVALID_ARG"
    assert loss_fwd(lib, total=S + 1) == "MOE_ERR_ALIGNMENT"
    assert loss_bwd(lib, dx=None, dW=None) == "MOE_ERR_INVALID_ARG"
    assert loss_bwd(lib, acc=3) == "MOE_ERR_INVALID_ARG"
    assert loss_bwd(lib, dw=9) == "MOE_ERR_DTYPE"
    assert loss_bwd(lib, dtype=F, dw=H) == "MOE_ERR_DTYPE"
    assert loss_bwd(lib, dloss=S + 2) == "MOE_ERR_ALIGNMENT"


def test_loss_workspace(lib):
    for dtype in (F, H):
        fwd, both = (pkg.moe_vocab_loss_workspace_size(8192, 2048, 50257, dtype, t) for t in (False, True))
        assert 0 < fwd <= both
        # in pieces: far less than the logits of a large batch
        assert pkg.moe_vocab_loss_workspace_size(1 << 17, 256, 1 << 17, dtype, True) < (1 << 34) * 2
    with pytest.raises(pkg.MoeError, match="SHAPE"):
        pkg.moe_vocab_loss_workspace_size(4, 7, 100, H, True)
    with pytest.raises(TypeError):
        pkg.vocab_loss_workspace(4, 8, 100, torch.float16, True, "cpu")


def test_bindings_check_shapes(lib):
    x, W = torch.zeros(4, 8), torch.zeros(10, 12)
    i = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(4)
    ws = torch.zeros(8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="W has shape"):
        pkg.moe_vocab_loss_fwd(x, W, i, f, f, ws)
    with pytest.raises(TypeError, match="W has type"):
        pkg.moe_vocab_loss_fwd(x.cuda() if torch.cuda.is_available() else x[:0], torch.zeros(10, 8, dtype=torch.bfloat16), i[:0], f[:0], f[:0], ws)
    with pytest.raises(ValueError, match="dh or dout"):
        pkg.moe_residual_norm_bwd(x, x, None, None, None, None, None, None, 1.0, 1.0, None, None, x, x, {}, False, ws)
    with pytest.raises(ValueError, match="unknown gradients"):
        pkg.moe_residual_norm_bwd(x, x, x, None, None, None, None, None, 1.0, 1.0, None, None, x, x, dict(dgama=f), False, ws)
    with pytest.raises(ValueError, match="gamma_post has"):
        pkg.moe_residual_norm_fwd(x, x, x, x, gamma_post=f)


# ----------------------------- the 64-bit forms --------------------------- #
def numeric(f, t, dy):
    """Central differences of sum(f() * dy) over the elements of t."""
    g = torch.zeros_like(t)
    flat, gf = t.view(-1), g.view(-1)
    for i in range(flat.numel()):
        v, h = flat[i].item(), 1e-5
        flat[i] = v + h
        up = (f() * dy).sum()
        flat[i] = v - h
        gf[i] = (up - (f() * dy).sum()) / (2 * h)
        flat[i] = v
    return g


@pytest.mark.parametrize("post,nxt", [(True, True), (False, True), (True, False)])
def test_join_reference_gradient_is_that_of_differences(post, nxt):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, y, gate, row = r(3, 5), r(3, 5), r(5), r(3)
    gp, gn = r(5) if post else None, r(5) if nxt else None
    dh, dout = r(3, 5) if nxt else None, r(3, 5)
    fwd = lambda: ref.join_fwd(x, y, gp, gn, gate, row, 0.8, 0.5, 1e-3)  # noqa: E731

    def f():
        out, h, _, _ = fwd()
        return torch.cat([out, h], 1) if nxt else out

    dy = torch.cat([dout, dh], 1) if nxt else dout
    out, _, ry, ro = fwd()
    got = ref.join_bwd(out, y, dh, dout, gp, gn, gate, row, 0.8, 0.5, ry, ro)
    for name, t in (("dx", x), ("dy", y), ("dgate", gate), ("drow_gate", row), ("dgamma_post", gp), ("dgamma_next", gn)):
        if t is not None:
            # differences of step 1e-5: truncation 1e-10 of third derivatives of order 10, roundings 1e-11
            assert torch.allclose(got[name], numeric(f, t, dy), atol=1e-7), name


def test_loss_reference_gradient_is_that_of_differences():
    g = torch.Generator().manual_seed(4)
    x, W = torch.randn(4, 3, generator=g, dtype=torch.float64), torch.randn(6, 3, generator=g, dtype=torch.float64)
    labels, dloss = torch.tensor([2, -100, 5, 0], dtype=torch.int32), torch.rand(4, generator=g, dtype=torch.float64)
    _, lse, _ = ref.loss_fwd(x, W, labels)
    dx, dW, _, _ = ref.loss_bwd(x, W, labels, lse, dloss)
    f = lambda: ref.loss_fwd(x, W, labels)[0]  # noqa: E731
    assert torch.allclose(dx, numeric(f, x, dloss), atol=1e-7) and torch.allclose(dW, numeric(f, W, dloss), atol=1e-7)
    assert (dx[1] == 0).all()
