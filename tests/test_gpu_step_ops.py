"""Operators that join blocks to a training step on the GPU against their 64-bit forms.

Tolerances, from the roundings.  U = 2^-24 is half a step of fp32, HALF[t] that
of a stored type.  A statistic of a row sums d positive squares: at most 16 a
thread and a tree over the threads, under 32 roundings, halved by the root, and
two or three more of the root and the products: STAT = 32 U.  Sums of terms of
either sign wander by the square root of their number: 64 U of the largest value
for up to 4096 comparable terms.
"""
import math

import pytest
import torch

import _step_ref as ref
import routing_permute_grouped_router_gb300 as pkg
from _util import check_no_device_error

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
STAT = 32 * U
F32_SUM = 64 * U
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module", autouse=True)
def built():
    from routing_permute_grouped_router_gb300 import build

    build.build()
    pkg.lib()
    torch.cuda.set_device(0)
    pkg.moe_get_device_error(clear=True)


def near(name, got, exp, rel=0.0, big=F32_SUM, tol=None):
    """|got - exp| <= (rel + half a step) |exp| + big max|exp| (or + tol), elementwise; both may hold the same NaN."""
    assert got.shape == exp.shape, f"{name}: {tuple(got.shape)} is not {tuple(exp.shape)}"
    if got.numel() == 0:
        return
    assert torch.equal(got.isnan(), exp.isnan()), f"{name}: NaN in other places"
    g, e = got.double().nan_to_num(0.0, 0.0, 0.0), exp.nan_to_num(0.0, 0.0, 0.0)
    room = (rel + HALF[got.dtype]) * e.abs() + (big * e.abs().max() if tol is None else tol)
    over = (g - e).abs() - room
    assert over.max() <= 0, f"{name}: off by {float((g - e).abs().max()):.3e} of {float(e.abs().max()):.3e}"


def rand(*shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# ----------------------------- residual path ------------------------------ #
def join_inputs(rows, d, t, post=True, nxt=True, gate=True, row=False, seed=1, branch=True):
    return dict(x=rand(rows, d, seed=seed, dtype=t), y=rand(rows, d, seed=seed + 1, dtype=t, scale=0.3) if branch else None,
                post=1 + rand(d, seed=seed + 2, scale=0.2) if post else None,
                nxt=1 + rand(d, seed=seed + 3, scale=0.2) if nxt else None,
                gate=rand(d, seed=seed + 4) if gate else None, row=rand(rows, seed=seed + 5) if row else None)


def run_fwd(i, rs=1.0, bs=1.0, eps=1e-6, stream=None, out=None, h=None):
    rows = i["x"].shape[0]
    nan = lambda like: torch.full_like(like, float("nan"))  # noqa: E731
    r = dict(out=nan(i["x"]) if out is None else out, h=None if i["nxt"] is None else nan(i["x"]) if h is None else h,
             ry=None if i["post"] is None else torch.full((rows,), float("nan"), device="cuda"),
             ro=None if i["nxt"] is None else torch.full((rows,), float("nan"), device="cuda"))
    pkg.moe_residual_norm_fwd(i["x"], i["y"], r["out"], r["h"], i["post"], i["nxt"], i["gate"], i["row"], rs, bs, eps,
                              r["ry"], r["ro"], stream)
    return r


def check_fwd(r, e):
    torch.cuda.synchronize()
    check_no_device_error()
    # the statistics' error, and sums of two terms that may cancel
    for name, v in zip(("out", "h", "ry", "ro"), e):
        if v is not None:
            near(name, r[name], v, rel=2 * STAT, big=8 * U)
        else:
            assert name not in r or r[name] is None


def run_bwd(i, f, dh, dout, rs, bs, accumulate=False, grads=None, dx=None, dy=None, ws=None):
    rows, d = i["x"].shape
    nan = lambda like: torch.full_like(like, float("nan"))  # noqa: E731
    if grads is None:
        grads = {}
        for n, on, size in (("dgamma_post", i["post"], d), ("dgamma_next", i["nxt"], d), ("dgate", i["gate"], d),
                            ("drow_gate", i["row"], rows)):
            if on is not None:
                grads[n] = torch.full((size,), float("nan"), device="cuda")
    dx = nan(i["x"]) if dx is None else dx
    dy = None if i["y"] is None else nan(i["x"]) if dy is None else dy
    ws = pkg.residual_norm_workspace(rows, d).fill_(255) if ws is None else ws
    pkg.moe_residual_norm_bwd(f["out"], i["y"], dh, dout, i["post"], i["nxt"], i["gate"], i["row"], rs, bs, f["ry"],
                              f["ro"], dx, dy, grads, accumulate, ws)
    return dict(dx=dx, dy=dy, **grads)


def check_bwd(r, e, add=None):
    torch.cuda.synchronize()
    check_no_device_error()
    for name, v in r.items():
        if v is not None:
            near(name, v, e[name] if add is None or name not in add else e[name] + add[name], rel=STAT)


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 8), (16, 4096), (33, 512), (129, 1000), (333, 2048), (7, 8192), (64, 520),
          (2, 8200), (3, 16384), (5, 9001), (1, 65536), (1030, 96), (4099, 1021), (9, 7001), (310, 6888), (700, 1007), (155, 8191),
          (17, 33), (1200, 31), (400, 2047)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_join(rows, d, dtype):
    i = join_inputs(rows, d, TYPES[dtype], row=rows % 2 == 1)
    r = run_fwd(i, 0.8, 0.5)
    check_fwd(r, ref.join_fwd(*i.values(), 0.8, 0.5))
    dh, dout = rand(rows, d, seed=8, dtype=TYPES[dtype]), rand(rows, d, seed=9, dtype=TYPES[dtype])
    e = ref.join_bwd(r["out"], i["y"], dh, dout, i["post"], i["nxt"], i["gate"], i["row"], 0.8, 0.5, r["ry"], r["ro"])
    b = run_bwd(i, r, dh, dout, 0.8, 0.5)
    check_bwd(b, e)
    again = run_bwd(i, r, dh, dout, 0.8, 0.5)
    assert all(torch.equal(b[n], again[n]) for n in b if b[n] is not None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [256, 1021, 8264])
@pytest.mark.parametrize("post,nxt,gate,row,branch,dout", [
    (True, True, True, True, True, True), (True, True, False, False, True, False), (False, True, True, False, True, True),
    (False, True, False, True, True, False), (True, False, True, True, True, True), (False, False, True, False, True, True),
    (False, False, False, False, True, True), (False, True, False, False, False, True),
    (False, True, False, False, False, False), (False, True, False, False, True, True)])
def test_join_parts(dtype, d, post, nxt, gate, row, branch, dout):
    rows, t = 77, TYPES[dtype]
    i = join_inputs(rows, d, t, post, nxt, gate, row, 21, branch)
    r = run_fwd(i, 1.0, 0.7)
    check_fwd(r, ref.join_fwd(*i.values(), 1.0, 0.7))
    dh = rand(rows, d, seed=8, dtype=t) if nxt else None
    do = rand(rows, d, seed=9, dtype=t) if dout else None
    e = ref.join_bwd(r["out"], i["y"], dh, do, i["post"], i["nxt"], i["gate"], i["row"], 1.0, 0.7, r["ry"], r["ro"])
    check_bwd(run_bwd(i, r, dh, do, 1.0, 0.7), e)
    if row:  # the row gate's gradient alone
        check_bwd(run_bwd(i, r, dh, do, 1.0, 0.7, grads=dict(drow_gate=torch.empty(rows, device="cuda"))), e)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(700, 512), (700, 1021), (40, 9000)])
def test_join_in_place_and_accumulated(rows, d, dtype):
    t = TYPES[dtype]
    i = join_inputs(rows, d, t, row=True, seed=31)
    a = run_fwd(i)
    for out, h in (("x", "y"), ("y", "x")):
        j = {n: None if v is None else v.clone() for n, v in i.items()}
        b = run_fwd(j, out=j[out], h=j[h])
        assert all(torch.equal(a[n], b[n]) for n in a)
    dh, dout = rand(rows, d, seed=8, dtype=t), rand(rows, d, seed=9, dtype=t)
    c = run_bwd(i, a, dh, dout, 1.0, 1.0)
    for dx, dy in ((0, 1), (1, 0)):
        given = [dh.clone(), dout.clone()]
        b = run_bwd(i, a, given[0], given[1], 1.0, 1.0, dx=given[dx], dy=given[dy])
        assert all(torch.equal(c[n], b[n]) for n in c)
    before = {n: torch.randn_like(c[n]) for n in ("dgamma_post", "dgamma_next", "dgate", "drow_gate")}
    b = run_bwd(i, a, dh, dout, 1.0, 1.0, True, {n: v.clone() for n, v in before.items()})
    for n in before:
        # one more rounding of the sum
        near(n, b[n], c[n].double() + (0 if n == "drow_gate" else before[n].double()), big=U)


def test_join_rows_of_zeros_and_non_finite_rows():
    """A row of zeros gives h = 0; a row with an infinity or a NaN keeps it to itself."""
    for t in TYPES.values():
        for d in (512, 1021, 9000):
            i = join_inputs(9, d, t, seed=41)
            i["x"][2], i["y"][2] = 0, 0
            i["y"][4, 3], i["x"][6, 5] = float("nan"), float("inf")
            r = run_fwd(i)
            e = ref.join_fwd(*i.values())
            ok = [0, 1, 2, 3, 5, 7, 8]
            for n, v in zip(("out", "h", "ry", "ro"), e):
                near(n, r[n][ok], v[ok], rel=2 * STAT, big=8 * U)
            assert (r["h"][2] == 0).all() and r["h"][4].isnan().all()
            torch.cuda.synchronize()


@pytest.mark.parametrize("d", [520, 1021, 1023, 4090, 9000])
def test_join_neighbours_of_a_row_do_not_reach_it(d):
    """Rows of NaN between the others: what copies bring of them beside a row is left out, and sums go by row."""
    for t in TYPES.values():
        i = join_inputs(641, d, t, seed=61, row=True)
        clean = {n: None if v is None else v.clone() for n, v in i.items()}
        i["x"][1::2], i["y"][1::2] = float("nan"), float("inf")
        r, e = run_fwd(i, 0.8, 0.5), run_fwd(clean, 0.8, 0.5)
        assert all(torch.equal(r[n][::2], e[n][::2]) for n in r)
        dh, dout = rand(641, d, seed=8, dtype=t), rand(641, d, seed=9, dtype=t)
        a = run_bwd(clean, e, dh, dout, 0.8, 0.5)
        dh[1::2], dout[1::2] = float("nan"), float("nan")
        b = run_bwd(i, r, dh, dout, 0.8, 0.5)
        for n in ("dx", "dy", "drow_gate"):
            assert torch.equal(a[n][::2], b[n][::2]), n
    torch.cuda.synchronize()


def test_join_no_rows():
    i = join_inputs(0, 64, torch.bfloat16)
    r = run_fwd(i)
    g = dict(dgamma_post=torch.ones(64, device="cuda"), dgamma_next=torch.ones(64, device="cuda"), dgate=torch.ones(64, device="cuda"))
    run_bwd(i, r, i["x"], i["x"], 1.0, 1.0, True, g)
    assert all((v == 1).all() for v in g.values())
    run_bwd(i, r, i["x"], i["x"], 1.0, 1.0, False, g)
    assert all((v == 0).all() for v in g.values())


def test_join_captured_and_on_another_stream():
    i = join_inputs(333, 2048, torch.bfloat16, row=True)
    dh, dout = rand(333, 2048, seed=8, dtype=torch.bfloat16), rand(333, 2048, seed=9, dtype=torch.bfloat16)
    a = run_fwd(i)
    c = run_bwd(i, a, dh, dout, 1.0, 1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, h, dx, dy = (torch.zeros_like(i["x"]) for _ in range(4))
    ry, ro = torch.zeros(333, device="cuda"), torch.zeros(333, device="cuda")
    grads = {n: torch.zeros_like(c[n]) for n in ("dgamma_post", "dgamma_next", "dgate", "drow_gate")}
    ws = pkg.residual_norm_workspace(333, 2048)

    def step():
        pkg.moe_residual_norm_fwd(i["x"], i["y"], out, h, i["post"], i["nxt"], i["gate"], i["row"], 1.0, 1.0, 1e-6, ry, ro)
        pkg.moe_residual_norm_bwd(out, i["y"], dh, dout, i["post"], i["nxt"], i["gate"], i["row"], 1.0, 1.0, ry, ro, dx, dy,
                                  grads, False, ws)

    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        for v in (out, h, dx, dy, ry, ro, *grads.values()):
            v.zero_()
        g.replay()
    s.synchronize()
    assert torch.equal(out, a["out"]) and torch.equal(h, a["h"]) and torch.equal(dx, c["dx"]) and torch.equal(dy, c["dy"])
    assert all(torch.equal(grads[n], c[n]) for n in grads)


def test_join_past_32_bits_of_elements():
    """More than 2^31 elements: the last rows."""
    rows, d, t = 530000, 4096, torch.bfloat16
    x = torch.zeros(rows, d, dtype=t, device="cuda")
    y = torch.zeros(rows, d, dtype=t, device="cuda")
    tail = join_inputs(5, d, t, seed=51)
    x[-5:], y[-5:] = tail["x"], tail["y"]
    h, out = torch.empty_like(x), torch.empty_like(x)
    pkg.moe_residual_norm_fwd(x, y, out, h, tail["post"], tail["nxt"], tail["gate"])
    e = ref.join_fwd(*tail.values())
    near("out", out[-5:], e[0], rel=2 * STAT, big=8 * U)
    near("h", h[-5:], e[1], rel=2 * STAT, big=8 * U)
    assert not out[:-5].any() and not h[:-5].any()


# ----------------------------- clipping ----------------------------------- #
NORM = 12 * U  # at most 16 squares to a sum in fp32, four sums added, halved by the root, rounded; the rest in 64 bits


def clip(src, dst, max_norm, norm=None):
    norm = torch.full((1,), float("nan"), device="cuda") if norm is None else norm
    l = pkg.grad_list(src, dst)
    pkg.moe_clip_grads(l, max_norm, norm, pkg.clip_workspace(len(src)).fill_(255))
    return float(norm[0])


def norm64(src):
    return math.sqrt(sum(float(t.double().square().sum()) for t in src))


def check_clip(src, max_norm, in_place):
    before = [t.clone() for t in src]
    n64 = norm64(src)
    dst = src if in_place else [torch.full_like(t, float("nan")) for t in src]
    n = clip(src, dst, max_norm)
    torch.cuda.synchronize()
    assert abs(n - n64) <= NORM * n64
    scale = min(1.0, max_norm / n64) if n64 > 0 else 1.0
    for b, t in zip(before, dst):
        near("clipped", t, b.double() * scale, rel=NORM + 2 * U, big=0.0)
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(before, src))


SIZES = [[1], [7], [4096], [32768 // 4], [32768 // 4 + 1], [3, 0, 5, 1021, 70001], [1000003], [0], [0, 0, 3], [17] * 97, [5, 9000] * 400]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "f32", "both"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_clip(sizes, kind, in_place):
    src = [rand(n, seed=60 + i, dtype=TYPES["bf16" if kind == "bf16" or (kind == "both" and i % 2) else "f32"]) for i, n in enumerate(sizes)]
    total = norm64(src)
    for ratio in (0.3, 2.0, math.inf):
        check_clip([t.clone() for t in src], ratio * total if total > 0 else 1.0, in_place)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_clip_views_at_any_offset(dtype):
    """Neighbours in one buffer: nothing between and around the tensors is touched."""
    t = TYPES[dtype]
    for first in range(9):
        for to in range(0, 9, 2):
            flat = rand(40000, seed=70 + first, dtype=t)
            out = torch.full_like(flat, 7.0)
            cuts = [(first, 31), (first + 40, 17000 + first), (first + 20000, 8), (first + 20008, 9)]
            src = [flat[a:a + n] for a, n in cuts]
            dst = [out[a - first + to:a - first + to + n] for a, n in cuts]
            total = norm64(src)
            assert abs(clip(src, dst, 0.5 * total) - total) <= NORM * total
            exp = torch.full((40000,), 7.0, dtype=torch.float64, device="cuda")
            for a, n in cuts:
                exp[a - first + to:a - first + to + n] = flat[a:a + n].double() * 0.5
            near("buffer", out, exp, rel=NORM + 2 * U, big=0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_clip_extreme_values(dtype):
    t = TYPES[dtype]
    x = rand(100000, seed=80, dtype=t)
    for scale in (2.0 ** 60, 2.0 ** 100, 2.0 ** -60, 2.0 ** -100):
        check_clip([(x.double() * scale).to(t), x.clone()], 0.25 * scale if scale > 1 else 1.0, False)
        check_clip([(x.double() * scale).to(t)], 100 * scale, False)
    tiny = torch.full((64,), 2.0 ** -130, device="cuda")  # subnormal float32
    assert abs(clip([tiny], None, 1.0) - 8 * 2.0 ** -130) <= 2.0 ** -149
    mixed = torch.zeros(70000, dtype=t, device="cuda")
    mixed[5], mixed[69999] = 3.0e38, -2.0 ** 100
    n64 = norm64([mixed])
    assert abs(clip([mixed], None, 1.0) - n64) <= NORM * n64


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("alone", [True, False])
def test_clip_of_what_is_not_finite(bad, alone):
    """Nothing is clipped, and the norm says why; a NaN among zeros counts too."""
    x = torch.zeros(50000, device="cuda") if alone else rand(50000, seed=90)
    x[40001] = bad
    y = rand(1000, seed=91, dtype=torch.bfloat16)
    out = [torch.empty_like(x), torch.empty_like(y)]
    n = clip([x, y], out, 0.5)
    assert math.isnan(n) if math.isnan(bad) else n == math.inf
    near("copy", out[0], x.double(), big=0.0)
    assert torch.equal(out[0].nan_to_num(1, 2, 3), x.nan_to_num(1, 2, 3)) and torch.equal(out[1], y)
    keep = x.clone()
    clip([x, y], [x, y], 0.5)
    assert torch.equal(x.nan_to_num(1, 2, 3), keep.nan_to_num(1, 2, 3))
    big = torch.full((4,), 3.0e38, device="cuda")  # each finite, their norm not
    assert clip([big], [big], 1.0) == math.inf and (big == 3.0e38).all()


def test_clip_nothing_and_partial_lists():
    assert clip([], None, 1.0) == 0.0
    z = torch.zeros(100, device="cuda")
    assert clip([z], [z], 1.0) == 0.0 and not z.any()
    a, b = rand(100, seed=1), rand(100, seed=2)
    out = torch.empty_like(b)
    n64 = norm64([a, b])
    assert abs(clip([a, b], [None, out], n64 / 4) - n64) <= NORM * n64
    near("second", out, b.double() / 4, rel=NORM + 2 * U, big=0.0)
    keep = a.clone()  # a norm of exactly max_norm is not past it
    three = torch.full((9,), 1.0, device="cuda")
    assert clip([three], [three], 3.0) == 3.0 and (three == 1).all() and torch.equal(a, keep)


def test_clip_is_deterministic_and_captured():
    src = [rand(n, seed=i) for i, n in enumerate((3000001, 17, 1 << 20))]
    out = [torch.empty_like(t) for t in src]
    l, norm, ws = pkg.grad_list(src, out), torch.zeros(1, device="cuda"), pkg.clip_workspace(3)
    pkg.moe_clip_grads(l, 1.0, norm, ws)
    first, copies = norm.clone(), [t.clone() for t in out]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pkg.moe_clip_grads(l, 1.0, norm, ws)
        norm.zero_()
        for t in out:
            t.zero_()
        g.replay()
    s.synchronize()
    assert torch.equal(norm, first) and all(torch.equal(a, b) for a, b in zip(out, copies))


def test_clip_past_32_bits_of_elements():
    n = (1 << 31) + 12345
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    x[-3:], x[0] = 4.0, 1.0
    assert abs(clip([x], [x], 3.5) - 7.0) <= NORM * 7
    assert (x[-3:] == 2.0).all() and x[0] == 0.5


# ----------------------------- vocabulary loss ---------------------------- #
def loss_inputs(T, d, V, t, ignored=0.0, seed=1, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = rand(V, d, seed=seed + 1, dtype=t, scale=d ** -0.5)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = (rand(T, d, seed=seed + 2, scale=scale) + 2 * W[labels].float()).to(t)
    labels[torch.randperm(T, generator=g, device="cuda")[:int(ignored * T)]] = -100
    return x, W, labels.int()


def logit_error(x, W):
    """Bound on the error of a logit.  At worst each group of 16 products is added with one truncation (2^-23 of the
    sum so far, itself at most the sum of magnitudes), after 16 more within the groups."""
    d = x.shape[1]
    return (d / 16 + 16) * 2.0 ** -23 * (x.double().abs() @ W.double().abs().t()).nan_to_num(0.0, 0.0, 0.0)


def run_loss(x, W, labels, total=True, ws=None):
    T, d = x.shape
    loss, lse = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    tot = torch.full((2,), float("nan"), device="cuda") if total else None
    ws = pkg.vocab_loss_workspace(T, d, W.shape[0], x.dtype, False).fill_(255) if ws is None else ws
    pkg.moe_vocab_loss_fwd(x, W, labels, loss, lse, ws, tot)
    return loss, lse, tot


def check_loss(x, W, labels):
    loss, lse, tot = run_loss(x, W, labels)
    torch.cuda.synchronize()
    check_no_device_error()
    e_loss, e_lse, _ = ref.loss_fwd(x, W, labels)
    valid = labels >= 0
    assert (loss[~valid] == 0).all() and (lse[~valid] == 0).all()
    if valid.any():
        ze = float(logit_error(x[valid], W).max())
        # two logits' errors, exp and log to 2 steps each and sums of V positive terms in a tree
        tol = 2 * ze + 64 * U
        near("lse", lse, e_lse, rel=4 * U, tol=tol)
        near("loss", loss, e_loss, rel=4 * U, tol=tol + 4 * U * float(e_lse.abs().max()))
        assert abs(float(tot[0]) - float(loss.double().sum())) <= 2 * U * float(loss.double().abs().sum())
    assert int(tot[1]) == int(valid.sum())
    return loss, lse


def run_loss_bwd(x, W, labels, lse, dloss, dw, accumulate=False, dx=True, dW=True, start=None, ws=None):
    T, d = x.shape
    gx = torch.full_like(x, float("nan")) if dx else None
    gW = None if not dW else torch.full(W.shape, float("nan"), dtype=dw, device="cuda") if start is None else start.clone()
    ws = pkg.vocab_loss_workspace(T, d, W.shape[0], x.dtype, True).fill_(255) if ws is None else ws
    pkg.moe_vocab_loss_bwd(x, W, labels, lse, dloss, gx, gW, accumulate, ws)
    return gx, gW


def check_loss_bwd(x, W, labels, lse, dloss, dw, start=None):
    gx, gW = run_loss_bwd(x, W, labels, lse, dloss, dw, start is not None, start=start)
    torch.cuda.synchronize()
    check_no_device_error()
    ex, eW, dz, at = ref.loss_bwd(x, W, labels, lse, dloss)
    if start is not None:
        eW = eW + start.double()
    assert (gx[(labels < 0)] == 0).all()
    if not len(at):
        assert torch.equal(gW.double(), eW)
        return gx, gW
    xs, Wd = x[at].double(), W.double()
    # dz: the logit's error times p, exp's, and its own rounding (8 bits for bf16 products, 16 for a float32 dW, 24)
    g = (torch.full((len(at),), 1.0 / len(at), device="cuda", dtype=torch.float64) if dloss is None else dloss[at].double())[:, None]
    p = dz.clone()
    p[torch.arange(len(at), device="cuda"), labels[at].long()] += g[:, 0]
    off = p.abs() * (2 * logit_error(xs, W) + 16 * U) + 8 * U * g.abs() * (p.abs() > 0.5 * g.abs())
    bf16 = x.dtype == torch.bfloat16
    steps = lambda n: (n / 16 + 16) * 2.0 ** -23  # noqa: E731
    for name, got, exp, bits, left, right in (
            ("dx", gx[at], ex[at], 2.0 ** -8 if bf16 else 2.0 ** -21, dz, Wd),
            ("dW", gW, eW, 2.0 ** -8 if dw == torch.bfloat16 else 2.0 ** -16 if bf16 else 2.0 ** -21, dz.t(), xs)):
        o = off if name == "dx" else off.t()
        room = (o + (bits + steps(left.shape[1])) * left.abs()) @ right.abs()
        near(name, got, exp, rel=4 * U, tol=room + 1e-38)
        # and together: the errors of single terms are independent, so they add as squares
        e = float((got.double() - exp).norm())
        half = HALF[got.dtype]
        most = (half + bits + 16 * U) * float(exp.norm()) + float((o @ right.abs()).norm())
        assert e <= most, f"{name}: {e:.3e} of {float(exp.norm()):.3e} together, {most:.3e} at most"
    return gx, gW


LOSSES = [(1, 64, 100), (1, 8, 1), (2, 8, 7), (5, 72, 257), (63, 64, 1000), (64, 128, 256), (65, 264, 255), (129, 1000, 5003),
          (257, 512, 777), (300, 2048, 1111), (17, 4096, 513), (1000, 64, 33), (40, 512, 40000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ignored", [0.0, 0.4])
@pytest.mark.parametrize("T,d,V", LOSSES)
def test_loss(T, d, V, ignored, dtype):
    x, W, labels = loss_inputs(T, d, V, TYPES[dtype], ignored, seed=T + V)
    _, lse = check_loss(x, W, labels)
    dloss = torch.rand(T, device="cuda") if T % 2 else None
    check_loss_bwd(x, W, labels, lse, dloss, torch.float32)
    if dtype == "bf16":
        check_loss_bwd(x, W, labels, lse, dloss, torch.bfloat16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_loss_every_token_count(dtype):
    for T in (1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 255, 256, 257):
        x, W, labels = loss_inputs(T, 136, 300, TYPES[dtype], 0.2, seed=T)
        _, lse = check_loss(x, W, labels)
        check_loss_bwd(x, W, labels, lse, None, torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 130])
def test_loss_ignored_tokens_may_hold_anything(dtype, T):
    x, W, labels = loss_inputs(T, 72, 500, TYPES[dtype], 0.5, seed=9)
    dloss = torch.rand(T, device="cuda")
    clean = x.clone()
    _, lse = check_loss(x, W, labels)
    a = check_loss_bwd(x, W, labels, lse, dloss, torch.float32)
    off = labels < 0
    labels[off] = torch.randint(-2 ** 31, -1, (int(off.sum()),), device="cuda", dtype=torch.int32)
    x[off], dloss[off] = float("nan"), float("inf")
    lse2 = lse.clone()
    lse2[off] = float("nan")
    loss, l2, _ = run_loss(x, W, labels)
    assert torch.equal(l2, lse) and (loss[off] == 0).all()
    b = run_loss_bwd(x, W, labels, lse2, dloss, torch.float32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 200])
def test_loss_all_ignored(dtype, T):
    x, W, labels = loss_inputs(T, 64, 300, TYPES[dtype])
    labels.fill_(-1)
    loss, lse, tot = run_loss(x, W, labels)
    assert not loss.any() and not lse.any() and not tot.any()
    for dw in (torch.float32, torch.bfloat16) if dtype == "bf16" else (torch.float32,):
        gx, gW = run_loss_bwd(x, W, labels, lse, None, dw)
        assert not gx.any() and not gW.any()
        start = rand(300, 64, seed=3, dtype=dw)
        gx, gW = run_loss_bwd(x, W, labels, lse, None, dw, True, start=start)
        assert not gx.any() and torch.equal(gW, start)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 300])
def test_loss_label_past_the_vocabulary_is_recorded(dtype, T):
    x, W, labels = loss_inputs(T, 64, 300, TYPES[dtype])
    labels[1] = 300
    loss, lse, tot = run_loss(x, W, labels)
    code, detail = pkg.moe_get_device_error(clear=True)
    assert pkg.STATUS[code] == "MOE_ERR_DEVICE_CHECK" and detail == (6 << 24) | 1
    assert loss[1] == 0 and lse[1] == 0 and int(tot[1]) == T - 1
    gx, gW = run_loss_bwd(x, W, labels, lse, None, torch.float32)
    assert pkg.moe_get_device_error(clear=True)[0] != 0
    keep = labels.clone()
    keep[1] = -1
    e = run_loss_bwd(x, W, keep, lse, None, torch.float32)
    assert torch.equal(gx, e[0]) and torch.equal(gW, e[1])
    check_no_device_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 150])
def test_loss_accumulated_and_one_sided(dtype, T):
    x, W, labels = loss_inputs(T, 264, 1003, TYPES[dtype], 0.1, seed=5)
    _, lse = check_loss(x, W, labels)
    for dw in (torch.float32, torch.bfloat16) if dtype == "bf16" else (torch.float32,):
        check_loss_bwd(x, W, labels, lse, None, dw, start=rand(1003, 264, seed=6, dtype=dw, scale=0.01))
        gx, gW = run_loss_bwd(x, W, labels, lse, None, dw)
        assert torch.equal(gx, run_loss_bwd(x, W, labels, lse, None, dw, dW=False)[0])
        assert torch.equal(gW, run_loss_bwd(x, W, labels, lse, None, dw, dx=False)[1])
        again = run_loss_bwd(x, W, labels, lse, None, dw)
        assert torch.equal(gx, again[0]) and torch.equal(gW, again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [9, 140])
def test_loss_large_logits(dtype, T):
    """Logits of thousands: the largest one alone counts; and logits all alike."""
    x, W, labels = loss_inputs(T, 64, 700, TYPES[dtype], seed=7, scale=3000.0)
    _, lse = check_loss(x, W, labels)
    x = torch.zeros_like(x)
    loss, lse = check_loss(x, W, labels)
    assert (lse - math.log(700)).abs().max() < 1e-5
    check_loss_bwd(x, W, labels, lse, None, torch.float32)


@pytest.mark.parametrize("T", [4, 150])
def test_loss_words_that_are_switched_off(T):
    """Rows of W of -inf, a whole tile of them and more: their logits are -inf and add nothing."""
    for t in TYPES.values():
        x, W, labels = loss_inputs(T, 64, 1500, t, seed=8)
        x = x.abs() + 0.01
        W[:600] = float("-inf")
        W[1400:] = float("-inf")
        labels = labels % 700 + 650
        loss, lse, _ = run_loss(x, W, labels)
        e_loss, e_lse, _ = ref.loss_fwd(x, W[600:1400], labels - 600)
        ze = float(logit_error(x, W[600:1400]).max())
        near("lse", lse, e_lse, rel=4 * U, tol=2 * ze + 64 * U)
        near("loss", loss, e_loss, rel=4 * U, tol=3 * ze + 64 * U)


def test_loss_non_finite_rows_stay_to_themselves():
    for t in TYPES.values():
        for T in (6, 140):
            x, W, labels = loss_inputs(T, 72, 400, t, seed=12)
            clean = run_loss(x, W, labels)
            x[3] = float("nan")
            loss, lse, _ = run_loss(x, W, labels)
            ok = [i for i in range(T) if i != 3]
            assert loss[3].isnan() and torch.equal(loss[ok], clean[0][ok]) and torch.equal(lse[ok], clean[1][ok])


# the float32 form of few tokens: groups of 8, 4, 2 and 1, the most of them and one token more, the longest rows and past them
@pytest.mark.parametrize("T,d,V", [(3, 4, 5), (8, 6656, 70), (9, 6660, 131), (24, 13312, 37), (25, 6660, 65), (13, 13316, 33), (24, 26624, 29),
                                   (25, 26624, 29), (48, 13312, 700), (49, 13312, 700), (5, 26628, 40), (12, 53248, 19), (13, 53248, 19), (2, 53252, 17), (1, 65536, 23), (41, 100, 9729), (48, 132, 4000), (49, 132, 4000)])
def test_loss_few_float32_tokens(T, d, V):
    x, W, labels = loss_inputs(T, d, V, torch.float32, 0.2, seed=T + d)
    labels[-1] = V - 1
    loss, lse = check_loss(x, W, labels)
    # an infinity counts as the largest bf16 here as with many tokens, and where it meets a zero adds nothing
    x[:, 1] = 0
    W[:, 1] = float("inf")
    W[V // 2, 0] = float("-inf")
    x[:, 0] = x[:, 0].abs() + 0.01
    labels[labels == V // 2] = 0
    loss, lse, _ = run_loss(x, W, labels)
    W[:, 1] = 0
    rest = [v for v in range(V) if v != V // 2]
    e_loss, e_lse, _ = ref.loss_fwd(x, W[rest], torch.where(labels > V // 2, labels - 1, labels))
    ze = float(logit_error(x, W[rest]).max())
    near("lse", lse, e_lse, rel=4 * U, tol=2 * ze + 64 * U)
    near("loss", loss, e_loss, rel=4 * U, tol=3 * ze + 64 * U)
    x[0] = float("nan")
    bad, bad_lse, _ = run_loss(x, W, labels)
    W[:, 1] = float("inf")
    again = run_loss(x, W, labels)
    assert torch.equal(bad_lse[1:], again[1][1:]) and torch.equal(bad[1:], again[0][1:])
    assert bad[0].isnan() if labels[0] >= 0 else bad[0] == 0
    check_no_device_error()


@pytest.mark.parametrize("dtype,T,d,V", [("bf16", 1024, 64, 300001), ("f32", 600, 64, 130003), ("bf16", 3000, 520, 50257)])
def test_loss_in_several_pieces(dtype, T, d, V):
    x, W, labels = loss_inputs(T, d, V, TYPES[dtype], 0.1, seed=13)
    loss, lse, _ = run_loss(x, W, labels)
    e_loss, e_lse, _ = ref.loss_fwd(x, W, labels)
    tol = 2 * float(logit_error(x[:64], W).max()) * 1.5 + 64 * U
    near("lse", lse, e_lse, rel=4 * U, tol=tol)
    near("loss", loss, e_loss, rel=4 * U, tol=tol)
    ex, eW, _, _ = ref.loss_bwd(x, W, labels, lse, None)
    for dw in (torch.float32, torch.bfloat16) if dtype == "bf16" else (torch.float32,):
        gx, gW = run_loss_bwd(x, W, labels, lse, None, dw)
        for got, exp, bits in ((gx, ex, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -19),
                               (gW, eW, 2.0 ** -8 if dw == torch.bfloat16 else 2.0 ** -16 if dtype == "bf16" else 2.0 ** -19)):
            # the roundings add as squares; 4 logit errors for p, of which the exponential makes a relative one
            rel = bits + HALF[got.dtype] + tol
            assert float((got.double() - exp).norm()) <= rel * float(exp.norm())
    torch.cuda.synchronize()
    check_no_device_error()


def test_loss_past_32_bits_of_elements():
    """x of more than 2^31 elements, most tokens ignored."""
    T, d, V = 530000, 4096, 500
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    labels = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    tx, W, tl = loss_inputs(300, d, V, torch.bfloat16, seed=14)
    x[-300:], labels[-300:] = tx, tl
    loss, lse, tot = run_loss(x, W, labels)
    e_loss, e_lse, _ = ref.loss_fwd(tx, W, tl)
    tol = 2 * float(logit_error(tx, W).max()) + 64 * U
    near("lse", lse[-300:], e_lse, rel=4 * U, tol=tol)
    near("loss", loss[-300:], e_loss, rel=4 * U, tol=tol)
    assert not loss[:-300].any() and int(tot[1]) == 300
    gx, gW = run_loss_bwd(x, W, labels, lse, None, torch.float32)
    ex, eW, _, _ = ref.loss_bwd(tx, W, tl, lse[-300:], None)
    assert not gx[:-300].any()
    assert float((gx[-300:].double() - ex).norm()) <= (2.0 ** -7 + tol) * float(ex.norm())
    assert float((gW.double() - eW).norm()) <= (2.0 ** -15 + tol) * float(eW.norm())
    check_no_device_error()


@pytest.mark.parametrize("T", [40, 70])
def test_loss_weights_past_32_bits_of_elements(T):
    d, V = 4096, 560000
    W = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    for i, part in enumerate(W.split(70000)):
        part.copy_(rand(part.shape[0], d, seed=100 + i, scale=d ** -0.5))
    x = rand(T, d, seed=99, dtype=torch.bfloat16)
    labels = torch.randint(V - 1000, V, (T,), device="cuda", dtype=torch.int32)
    loss, lse, _ = run_loss(x, W, labels)
    z = torch.cat([x.double() @ part.double().t() for part in W.split(70000)], 1)
    e_lse = torch.logsumexp(z, 1)
    tol = 2 * float(logit_error(x, W[:4096]).max()) * 1.5 + 64 * U
    near("lse", lse, e_lse, rel=4 * U, tol=tol)
    near("loss", loss, e_lse - z.gather(1, labels.long()[:, None])[:, 0], rel=4 * U, tol=tol)
    dz = torch.exp(z - lse.double()[:, None])
    dz[torch.arange(T, device="cuda"), labels.long()] -= 1
    dz /= T
    gx, gW = run_loss_bwd(x, W, labels, lse, None, torch.bfloat16)
    for at in (0, V - 3000):
        e = dz[:, at:at + 3000].t() @ x.double()
        assert float((gW[at:at + 3000].double() - e).norm()) <= (2.0 ** -7 + tol) * float(e.norm())
    e = sum(a @ b.double() for a, b in zip(dz.split(70000, 1), W.split(70000)))
    assert float((gx.double() - e).norm()) <= (2.0 ** -7 + tol) * float(e.norm())
    check_no_device_error()


@pytest.mark.parametrize("T", [8, 300])
def test_loss_captured_and_on_another_stream(T):
    x, W, labels = loss_inputs(T, 512, 2000, torch.bfloat16, 0.2, seed=15)
    loss, lse, tot = run_loss(x, W, labels)
    gx, gW = run_loss_bwd(x, W, labels, lse, None, torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = [torch.zeros_like(v) for v in (loss, lse, tot, gx, gW)]
    ws = pkg.vocab_loss_workspace(T, 512, 2000, torch.bfloat16, True)

    def step():
        pkg.moe_vocab_loss_fwd(x, W, labels, o[0], o[1], ws, o[2])
        pkg.moe_vocab_loss_bwd(x, W, labels, o[1], None, o[3], o[4], False, ws)

    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        for v in o:
            v.zero_()
        g.replay()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, (loss, lse, tot, gx, gW)))


# ----------------------------- all of them -------------------------------- #
def test_step_ops_from_new_threads():
    """Several host threads whose first CUDA calls these are, each on a stream of its own."""
    import threading

    i = join_inputs(300, 520, torch.bfloat16, seed=71)
    x, W, labels = loss_inputs(300, 520, 1000, torch.bfloat16, 0.1, seed=72)
    src = [rand(5000, seed=73)]
    torch.cuda.synchronize()
    got, failed = {}, []

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                a = run_fwd(i)
                b = run_bwd(i, a, i["x"], i["y"], 1.0, 1.0)
                loss, lse, _ = run_loss(x, W, labels)
                few, _, _ = run_loss(x[:20].contiguous(), W, labels[:20].contiguous())
                g = run_loss_bwd(x, W, labels, lse, None, torch.float32)
                out = [torch.empty_like(src[0])]
                norm = torch.zeros(1, device="cuda")
                pkg.moe_clip_grads(pkg.grad_list(src, out), 1.0, norm, pkg.clip_workspace(1))
            s.synchronize()
            got[k] = [a["out"], a["h"], b["dx"], b["dy"], b["dgate"], loss, lse, few, *g, norm, *out]
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for k in range(1, 4):
        assert all(torch.equal(a, b) for a, b in zip(got[0], got[k]))
    check_no_device_error()


def test_step_ops_refuse_views_types_and_places():
    x = rand(8, 64, seed=1, dtype=torch.bfloat16)
    g, f, i32 = rand(64, seed=2), rand(8, seed=3), torch.zeros(8, dtype=torch.int32, device="cuda")
    wide = rand(8, 128, seed=4, dtype=torch.bfloat16)
    W, ws = rand(100, 64, seed=5, dtype=torch.bfloat16), pkg.vocab_loss_workspace(8, 64, 100, torch.bfloat16, True)
    with pytest.raises(ValueError, match="contiguous"):
        pkg.moe_residual_norm_fwd(x, wide[:, ::2], x.clone(), None)
    with pytest.raises(TypeError, match="y has type"):
        pkg.moe_residual_norm_fwd(x, x.float(), x.clone(), None)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.moe_residual_norm_fwd(x, x.cpu(), x.clone(), None)
    with pytest.raises(ValueError, match="gate has"):
        pkg.moe_residual_norm_fwd(x, x.clone(), x.clone(), None, gate=f)
    flat = rand(8 * 64 + 8, seed=6, dtype=torch.bfloat16)
    with pytest.raises(pkg.MoeError, match="ALIGNMENT"):
        pkg.moe_residual_norm_fwd(flat[1:513].view(8, 64), x, x.clone(), None)
    with pytest.raises(TypeError, match="labels has type"):
        pkg.moe_vocab_loss_fwd(x, W, i32.long(), f, f.clone(), ws)
    with pytest.raises(ValueError, match="labels has"):
        pkg.moe_vocab_loss_fwd(x, W, i32[:7], f, f.clone(), ws)
    with pytest.raises(ValueError, match="contiguous"):
        pkg.moe_vocab_loss_fwd(x, rand(64, 100, seed=7, dtype=torch.bfloat16).t(), i32, f, f.clone(), ws)
    with pytest.raises(pkg.MoeError, match="WORKSPACE"):
        pkg.moe_vocab_loss_bwd(x, W, i32, f, None, x.clone(), None, False, ws[:1000])
    with pytest.raises(TypeError, match="dW has type"):
        pkg.moe_vocab_loss_bwd(x, W, i32, f, None, None, W.half(), False, ws)
    with pytest.raises(ValueError, match="contiguous"):
        pkg.grad_list([wide[:, :3]])
    with pytest.raises(pkg.MoeError, match="INVALID_ARG"):
        pkg.moe_clip_grads(pkg.grad_list([g, g], [g, g]), 1.0, f[:1].clone(), pkg.clip_workspace(2))
    check_no_device_error()
