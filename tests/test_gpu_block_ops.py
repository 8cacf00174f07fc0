"""Operators around the layer on the GPU against their 64-bit forms.

Tolerances.  A bf16 output carries one rounding, at most 2^-9 of the element
(half an ulp of 8 significant bits); 2^-8 leaves room for a sum that falls on
the other side of a tie.  fp32 sums of up to 4096 comparable terms wander by
sqrt(4096) roundings of 2^-24: 64 * 2^-24 of the tensor's largest value.  In
the few-token layer h is held in at least 16 bits: 2^-16 of the largest value
for bf16 layers.
"""
import numpy as np
import pytest
import torch

import _block_ref as ref
import routing_permute_grouped_router_gb300 as pkg
from _util import check_no_device_error, to64
from oracle import moe_oracle as O
from routing_permute_grouped_router_gb300 import layer
from routing_permute_grouped_router_gb300 import workload as W

pytestmark = pytest.mark.gpu
LS = W.LayerShape
F32_SUM = 64 * 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    from routing_permute_grouped_router_gb300 import build

    build.build()
    pkg.lib()
    torch.cuda.set_device(0)
    pkg.moe_get_device_error(clear=True)


def near(name, got, exp, rel=0.0, big=F32_SUM):
    """|got - exp| <= rel |exp| + big max|exp|, elementwise."""
    if isinstance(got, torch.Tensor):
        rel = 2.0 ** -8 if got.dtype == torch.bfloat16 else rel
    g, e = to64(got), np.asarray(exp, np.float64)
    assert g.shape == e.shape, f"{name}: shape {g.shape} != {e.shape}"
    assert np.isfinite(g).all(), f"{name}: non-finite values"
    if e.size:
        over = np.abs(g - e) - (rel * np.abs(e) + big * np.abs(e).max())
        assert over.max() <= 0, f"{name}: off by {np.abs(g - e).max():.3e} of {np.abs(e).max():.3e}"


# ----------------------------- few-token layer ---------------------------- #
def decode(wl, T, residual=None, stream=None, capacity=-1):
    s = wl.shape
    cfg = pkg.config(T, s.d_model, s.d_ff, s.E, s.k, s.capacity_factor, capacity,
                     pkg.MOE_BF16 if s.dtype == W.BF16 else pkg.MOE_F32)
    w = dict(W_r=torch.from_numpy(wl.W_r).cuda(), bias=None if wl.bias is None else torch.from_numpy(wl.bias).cuda(),
             W1=wl.W1.torch("cuda"), W3=wl.W3.torch("cuda"), W2=wl.W2.torch("cuda"))
    x = wl.x[0].torch("cuda")[:T].contiguous()
    y = torch.full_like(x, float("nan"))
    ids = torch.full((T, s.k), -7, dtype=torch.int32, device="cuda")
    gates = torch.full((T, s.k), -7.0, device="cuda")
    ws = pkg.decode_workspace(cfg).fill_(255)  # nothing in it may be relied on
    pkg.moe_layer_decode(cfg, w, x, residual, y, ids, gates, ws, stream)
    return dict(cfg=cfg, w=w, x=x, y=y, ids=ids, gates=gates, ws=ws)


def decode_ref(wl, T, C=None):
    s = wl.shape
    return O.forward(wl.x[0].f64()[:T], wl.W_r, wl.bias, wl.W1.f64(), wl.W3.f64(), wl.W2.f64(), s.k, C)


def check_decode(r, e, residual=None):
    torch.cuda.synchronize()
    check_no_device_error()
    assert np.array_equal(r["ids"].cpu().numpy(), e["ids"])
    near("gates", r["gates"], e["gates"], big=1e-6)
    y = e["y"] if residual is None else e["y"] + to64(residual)
    near("y", r["y"], y, big=2.0 ** -16 if r["y"].dtype == torch.bfloat16 else F32_SUM)


DECODE = [
    LS("one_token", 1, 512, 256, 32, 4, 0.0, W.BF16, zipf_s=1.3),
    LS("one_expert", 64, 256, 256, 1, 1, 0.0, W.BF16),
    LS("every_pick", 64, 256, 512, 8, 8, 0.0, W.BF16),
    LS("capacity_one", 33, 512, 256, 64, 2, 1.0, W.BF16, zipf_s=1.1),
    LS("odd_counts", 47, 768, 512, 7, 3, 1.25, W.BF16),
    LS("e128", 64, 256, 256, 128, 8, 0.0, W.BF16),
    LS("wide", 17, 4096, 256, 4, 2, 0.0, W.BF16, zipf_s=2.0),
    LS("long_f", 16, 256, 4096, 5, 2, 0.0, W.BF16),
    LS("f32_one_token", 1, 64, 128, 4, 1, 1.25, W.F32),
    LS("f32_odd", 33, 100, 36, 7, 3, 1.0, W.F32, zipf_s=1.1),
    LS("f32_tiny", 3, 4, 4, 3, 2, 0.0, W.F32),
    LS("f32_wide", 64, 1000, 516, 3, 2, 0.0, W.F32, zipf_s=2.0),
    LS("f32_e128", 64, 132, 260, 128, 8, 0.0, W.F32),
]


@pytest.mark.parametrize("shape", DECODE, ids=lambda s: s.name)
def test_decode(shape):
    wl = W.make(shape, seed=11, micro_batches=1, with_dy=False)
    T = shape.T
    C = O.capacity(T, shape.k, shape.E, shape.capacity_factor)
    e = decode_ref(wl, T, C)
    check_decode(decode(wl, T), e)
    res = torch.randn(T, shape.d_model, device="cuda").to(TYPES["bf16" if shape.dtype == W.BF16 else "f32"])
    r = decode(wl, T, res)
    check_decode(r, e, res)
    first = r["y"].clone()  # the same again, in the workspace as it was left
    pkg.moe_layer_decode(r["cfg"], r["w"], r["x"], res, r["y"], r["ids"], r["gates"], r["ws"])
    assert torch.equal(first, r["y"])


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_decode_every_token_count(dtype):
    s = LS("any", 64, 256, 256, 6, 2, 0.0, dtype, zipf_s=1.0)
    wl = W.make(s, seed=5, micro_batches=1, with_dy=False)
    for T in (1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64):
        check_decode(decode(wl, T), decode_ref(wl, T))


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("capacity", [0, 1, 3])
def test_decode_capacity(dtype, capacity):
    """Capacity 0 drops every pick: y is the residual, or 0."""
    s = LS("cap", 20, 256, 512, 4, 2, 0.0, dtype)
    wl = W.make(s, seed=6, micro_batches=1, with_dy=False)
    e = decode_ref(wl, 20, capacity)
    if capacity == 0:
        assert not e["y"].any()
    check_decode(decode(wl, 20, capacity=capacity), e)
    res = torch.randn(20, 256, device="cuda").to(torch.bfloat16 if dtype == W.BF16 else torch.float32)
    check_decode(decode(wl, 20, res, capacity=capacity), e, res)


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_decode_bad_values_stay_where_they_are(dtype):
    """A token of NaN or infinity spoils its own row alone, and experts nobody picks are not read."""
    s = LS("bad", 24, 256, 256, 8, 2, 0.0, dtype)
    wl = W.make(s, seed=7, micro_batches=1, with_dy=False)
    e = decode_ref(wl, 24)
    r = decode(wl, 24)
    for v in (float("nan"), float("inf")):
        x = r["x"].clone()
        x[5, 3] = v
        y = torch.empty_like(x)
        pkg.moe_layer_decode(r["cfg"], r["w"], x, None, y, r["ids"], r["gates"], r["ws"])
        torch.cuda.synchronize()
        check_no_device_error()
        assert not torch.isfinite(y[5]).any()
        ok = [t for t in range(24) if t != 5]
        near("y", y[ok], e["y"][ok], big=2.0 ** -16 if dtype == W.BF16 else F32_SUM)
        ids = r["ids"].cpu().numpy()
        assert ids.min() >= 0 and ids.max() < 8
    one = decode(wl, 1)
    unpicked = [i for i in range(8) if i not in e["ids"][0]]
    for n in ("W1", "W3", "W2"):
        one["w"][n][unpicked] = float("nan")
    y = torch.empty_like(one["x"])
    pkg.moe_layer_decode(one["cfg"], one["w"], one["x"], None, y, None, None, one["ws"])
    near("y", y, e["y"][:1], big=2.0 ** -16 if dtype == W.BF16 else F32_SUM)


def test_decode_no_tokens_and_side_stream():
    s = LS("side", 9, 256, 256, 4, 2, 0.0, W.BF16)
    wl = W.make(s, seed=8, micro_batches=1, with_dy=False)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        r = decode(wl, 9, stream=st)
    st.synchronize()
    check_decode(r, decode_ref(wl, 9))
    cfg = pkg.config(0, 256, 256, 4, 2)
    empty = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    n0 = pkg.moe_launch_count()
    pkg.moe_layer_decode(cfg, r["w"], empty, None, empty, None, None, r["ws"])
    assert pkg.moe_launch_count() == n0


# ----------------------------- layer norm --------------------------------- #
NORM = [(1, 1), (3, 2), (7, 129), (5, 1000), (1000, 256), (333, 2048), (40, 4095), (64, 4096), (9, 8192), (5, 8193),
        (3, 20000), (2, 65536), (700, 8), (2000, 60)]


def norm_inputs(rows, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(rows, d) * (0.5 + torch.rand(rows, 1, generator=g, device="cuda")) + 0.3 * r(rows, 1)).to(TYPES[dtype])
    return x, r(rows, d).to(TYPES[dtype]), r(rows, d).to(TYPES[dtype]), 1 + 0.2 * r(d), 0.1 * r(d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", NORM)
def test_norm(rows, d, dtype):
    x, dy, res, gamma, beta = norm_inputs(rows, d, dtype)
    eps = 1e-5
    f = dict(dtype=torch.float32, device="cuda")
    y, mean, rstd = torch.full_like(x, float("nan")), torch.empty(rows, **f), torch.empty(rows, **f)
    pkg.moe_norm_fwd(x, gamma, beta, eps, y, mean, rstd)
    x64, dy64, g64 = to64(x), to64(dy), to64(gamma)
    ey, emean, erstd = ref.norm_fwd(x64, g64, to64(beta), eps)
    near("y", y, ey)
    near("mean", mean, emean)
    near("rstd", rstd, erstd)
    y2 = torch.empty_like(x)
    pkg.moe_norm_fwd(x, gamma, beta, eps, y2)  # without the statistics
    assert torch.equal(y, y2)

    # a row of one element (d = 1) has x = mean: rstd = 1 / sqrt(eps), dx = 0 exactly
    edx, edg, edb = ref.norm_bwd(x64, dy64, g64, to64(mean), to64(rstd))
    ws = pkg.norm_workspace(rows, d).fill_(255)
    dx = torch.full_like(x, float("nan"))
    dg, db = torch.full((d,), 3.0, device="cuda"), torch.full((d,), -2.0, device="cuda")
    pkg.moe_norm_bwd(x, dy, gamma, mean, rstd, None, dx, dg, db, False, ws)
    # terms of dx are up to rstd |v|: the tensor's largest value may cancel below them (d = 1, 2)
    big = F32_SUM * max(1.0, np.abs(to64(rstd)[:, None] * dy64 * g64).max() / max(np.abs(edx).max(), 1e-30))
    if np.abs(edx).max() > 0:
        near("dx", dx, edx, big=big)
    near("dgamma", dg, edg, big=F32_SUM if np.abs(edg).max() > 0 else 0)
    near("dbeta", db, edb)
    # added to what is there, with the residual branch's gradient
    pkg.moe_norm_bwd(x, dy, gamma, mean, rstd, res, dx, dg, db, True, ws)
    near("dx + dres", dx, edx + to64(res), big=max(big * np.abs(edx).max() / np.abs(edx + to64(res)).max(), F32_SUM))
    near("2 dgamma", dg, 2 * edg)
    near("2 dbeta", db, 2 * edb)
    check_no_device_error()


def test_norm_gradient_against_differences():
    """Directional derivatives of the 64-bit forward at the fp32 inputs: truncation e^2, far below the fp32 sums."""
    x, dy, _, gamma, beta = norm_inputs(13, 96, "f32", 2)
    u = np.random.default_rng(1).standard_normal((13, 96))
    ug = np.random.default_rng(2).standard_normal(96)
    f = dict(dtype=torch.float32, device="cuda")
    y, mean, rstd, dx = torch.empty_like(x), torch.empty(13, **f), torch.empty(13, **f), torch.empty_like(x)
    dg, db = torch.empty(96, **f), torch.empty(96, **f)
    pkg.moe_norm_fwd(x, gamma, beta, 1e-5, y, mean, rstd)
    pkg.moe_norm_bwd(x, dy, gamma, mean, rstd, None, dx, dg, db, False, pkg.norm_workspace(13, 96))

    def loss(s, sg, sb):
        return (ref.norm_fwd(to64(x) + s * u, to64(gamma) + sg * ug, to64(beta) + sb * ug, 1e-5)[0] * to64(dy)).sum()

    e = 1e-4
    for (a, b, c), got, along in (((e, 0, 0), dx, u), ((0, e, 0), dg, ug), ((0, 0, e), db, ug)):
        want = (loss(a, b, c) - loss(-a, -b, -c)) / (2 * e)
        terms = np.abs(to64(got) * along).sum()
        assert abs((to64(got) * along).sum() - want) <= F32_SUM * terms + 1e-6


def test_norm_large_mean_and_constant_rows():
    """A mean of 1000 times the deviation does not cancel; a constant row has variance 0 and y = beta."""
    x = torch.randn(6, 512, device="cuda") + 1000.0
    x[3] = 7.0
    gamma, beta = torch.randn(512, device="cuda"), torch.randn(512, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    pkg.moe_norm_fwd(x, gamma, beta, 1e-5, y, mean, rstd)
    ey, _, erstd = ref.norm_fwd(to64(x), to64(gamma), to64(beta), 1e-5)
    # the mean's own rounding, 2^-24 of 1000 and the sum's, moves every element of a row alike
    move = 512 ** 0.5 * 2.0 ** -24 * 1000
    ok = [0, 1, 2, 4, 5]
    assert np.abs(to64(y) - ey)[ok].max() <= 2 * move * np.abs(to64(gamma)).max()
    assert torch.equal(y[3], beta)
    near("rstd", rstd[ok], erstd[ok])


def test_norm_in_place_no_rows_and_bad_rows():
    x, dy, res, gamma, beta = norm_inputs(50, 1024, "bf16", 4)
    y, mean, rstd = torch.empty_like(x), torch.empty(50, device="cuda"), torch.empty(50, device="cuda")
    pkg.moe_norm_fwd(x, gamma, beta, 1e-5, y, mean, rstd)
    z = x.clone()
    pkg.moe_norm_fwd(z, gamma, beta, 1e-5, z)
    assert torch.equal(y, z)
    ws, dg, db = pkg.norm_workspace(50, 1024), torch.empty(1024, device="cuda"), torch.empty(1024, device="cuda")
    dx = torch.empty_like(x)
    pkg.moe_norm_bwd(x, dy, gamma, mean, rstd, res, dx, dg, db, False, ws)
    z = res.clone()
    pkg.moe_norm_bwd(x, dy, gamma, mean, rstd, z, z, dg, db, False, ws)
    assert torch.equal(dx, z)
    # a row of NaN spoils its own row of y
    x[7, 9] = float("nan")
    pkg.moe_norm_fwd(x, gamma, beta, 1e-5, z)
    assert torch.isnan(z[7]).all() and torch.equal(z[:7], y[:7]) and torch.equal(z[8:], y[8:])
    # no rows: nothing to write but the gradients' zeros
    none = x[:0]
    pkg.moe_norm_fwd(none, gamma, beta, 1e-5, none)
    pkg.moe_norm_bwd(none, none, gamma, mean[:0], rstd[:0], None, none, dg, db, False, ws)
    assert not dg.any() and not db.any()


@pytest.mark.parametrize("d", [64, 1021, 16384])
def test_norm_weights_at_any_address(d):
    """gamma, beta and the statistics need no more than their own alignment."""
    x, dy, _, gamma, beta = norm_inputs(6, d, "bf16", 6)
    v = torch.empty(4 * d + 9, device="cuda")
    g2, b2 = v[1:d + 1], v[d + 2:2 * d + 2]
    g2.copy_(gamma), b2.copy_(beta)
    dg2, db2 = v[2 * d + 3:3 * d + 3], v[3 * d + 4:4 * d + 4]
    dg, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    out = []
    for g, b, p, q in ((gamma, beta, dg, db), (g2, b2, dg2, db2)):
        y, mean, rstd, dx = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda"), torch.empty_like(x)
        pkg.moe_norm_fwd(x, g, b, 1e-5, y, mean, rstd)
        pkg.moe_norm_bwd(x, dy, g, mean, rstd, None, dx, p, q, False, pkg.norm_workspace(6, d))
        out.append((y, dx, p.clone(), q.clone()))
    for s, t in zip(*out):  # the wide kernels sum in another order there
        assert torch.equal(s, t) if d <= 8192 else (s.float() - t.float()).abs().max() <= 2 ** -7 * s.float().abs().max()


def test_norm_past_32_bit_offsets():
    rows, d = 300000, 8192  # 2.46e9 elements
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(5, d, device="cuda").bfloat16()
    x[-5:] = tail
    gamma, beta = torch.randn(d, device="cuda"), torch.randn(d, device="cuda")
    y = torch.empty_like(x)
    pkg.moe_norm_fwd(x, gamma, beta, 1e-5, y)
    near("y", y[-5:], ref.norm_fwd(to64(tail), to64(gamma), to64(beta), 1e-5)[0])


# ----------------------------- dropout ------------------------------------ #
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 1000, 4096 * 33 + 5])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.97])
def test_dropout(n, p, dtype):
    y, res = (torch.randn(n, device="cuda").to(TYPES[dtype]) for _ in range(2))
    seed, offset = 0xFEDCBA9876543210, 0x123456789ABCDEF1
    e = ref.dropout(to64(y), p, seed, offset)
    out = torch.empty_like(y)
    pkg.moe_dropout_add(y, res, out, p, seed, offset)
    near("out", out, e + to64(res), rel=2.0 ** -22, big=2.0 ** -22)
    pkg.moe_dropout_add(y, None, out, p, seed, offset)
    near("out", out, e, rel=2.0 ** -22, big=0)
    assert np.array_equal(to64(out) != 0, (e != 0))
    dy = torch.empty_like(y)
    pkg.moe_dropout_bwd(y, dy, p, seed, offset)  # the same mask
    assert torch.equal(out, dy)
    z = y.clone()
    pkg.moe_dropout_add(z, res, z, p, seed, offset)
    pkg.moe_dropout_add(y, res, out, p, seed, offset)
    assert torch.equal(z, out)
    z = res.clone()
    pkg.moe_dropout_add(y, z, z, p, seed, offset)
    assert torch.equal(z, out)


def test_dropout_rate_and_independence():
    n, p = 1 << 22, 0.3
    one, out = torch.ones(n, device="cuda"), torch.empty(n, device="cuda")
    keeps = []
    for seed, offset in ((1, 0), (1, 1), (2, 0)):
        pkg.moe_dropout_add(one, None, out, p, seed, offset)
        keeps.append((out != 0).double())
        # five standard deviations of n draws; p itself to within 2^-17
        assert abs(keeps[-1].mean().item() - (1 - p)) < 5 * (p * (1 - p) / n) ** 0.5 + 2.0 ** -17
    for i, j in ((0, 1), (0, 2), (1, 2)):
        cov = (keeps[i] * keeps[j]).mean().item() - keeps[i].mean().item() * keeps[j].mean().item()
        assert abs(cov) < 5 * p * (1 - p) / n ** 0.5


def test_dropout_of_bad_values_is_zero():
    y = torch.full((4096,), float("nan"), device="cuda")
    y[::2] = float("inf")
    out, res = torch.empty_like(y), torch.randn(4096, device="cuda")
    pkg.moe_dropout_add(y, res, out, 0.5, 3, 4)
    keep = ref.draws(0, 4096, 3, 4) >= ref.cut_of(0.5)
    got = out.cpu().numpy()
    assert np.array_equal(got[~keep], res.cpu().numpy()[~keep]) and not np.isfinite(got[keep]).any()


def test_dropout_past_32_bit_offsets():
    n = (1 << 32) + 1003
    y = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    pkg.moe_dropout_bwd(y, y, 0.25, 5, 6)
    first = n - 3001
    e = ref.dropout(np.ones(3001), 0.25, 5, 6, first)
    near("tail", y[first:], e)


# ----------------------------- together ----------------------------------- #
def block_ref(wl, x, gamma, beta, eps, p, seed, offset):
    s = wl.shape
    h, mean, rstd = ref.norm_fwd(x, gamma, beta, eps)
    C = O.capacity(x.shape[0], s.k, s.E, s.capacity_factor)
    st = O.forward(h, wl.W_r, wl.bias, wl.W1.f64(), wl.W3.f64(), wl.W2.f64(), s.k, C)
    return h, mean, rstd, st, x + ref.dropout(st["y"], p, seed, offset)


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_block_forward_backward_and_decode(dtype):
    """The whole sub-block; its layer's products round to bf16 (the layer's own tolerance, 2e-2 or 1e-4 of the
    largest value)."""
    s = LS("block", 40, 256, 512, 4, 2, 1.25, dtype, backward=True)
    wl = W.make(s, seed=21, micro_batches=1, with_dy=True)
    L = layer.from_workload(wl)
    g = np.random.default_rng(9)
    gamma, beta = (1 + 0.1 * g.standard_normal(256)).astype(np.float32), (0.1 * g.standard_normal(256)).astype(np.float32)
    blk = layer.MoEBlock(L, torch.from_numpy(gamma).cuda(), torch.from_numpy(beta).cuda(), p=0.2)
    x, dout = wl.x[0].torch("cuda"), wl.dy[0].torch("cuda")
    x64, dout64 = wl.x[0].f64(), wl.dy[0].f64()
    out = blk.forward(x, seed=4, offset=77).clone()
    dx = blk.backward(x, dout, False, seed=4, offset=77)
    torch.cuda.synchronize()
    check_no_device_error()
    h, mean, rstd, st, eout = block_ref(wl, x64, gamma.astype(np.float64), beta.astype(np.float64), 1e-5, 0.2, 4, 77)
    assert np.array_equal(L.saved["ids"].cpu().numpy(), st["ids"])  # no pick is near enough for norm(x)'s rounding
    tol = 2e-2 if dtype == W.BF16 else 1e-4

    def close(name, got, exp):
        assert np.abs(to64(got) - exp).max() <= tol * np.abs(exp).max(), name

    close("out", out, eout)
    gr = O.backward(ref.dropout(dout64, 0.2, 4, 77), h, wl.W_r, wl.W1.f64(), wl.W3.f64(), wl.W2.f64(), st)
    edx, edg, edb = ref.norm_bwd(x64, gr["dx"], gamma.astype(np.float64), mean, rstd)
    close("dx", dx, edx + dout64)
    close("dgamma", blk.dgamma, edg)
    close("dbeta", blk.dbeta, edb)
    close("dW1", L.grads["dW1"], gr["dW1"])
    for T in (1, 5, 40):  # the serving step: no dropout, capacity of its own T
        close("decode", blk.decode(x[:T]), block_ref(wl, x64[:T], gamma.astype(np.float64), beta.astype(np.float64),
                                                     1e-5, 0.0, 0, 0)[4])
    check_no_device_error()


def test_block_decode_in_a_graph():
    s = LS("graph", 8, 512, 256, 8, 2, 0.0, W.BF16)
    wl = W.make(s, seed=22, micro_batches=1, with_dy=False)
    L = layer.from_workload(wl, training=False)
    blk = layer.MoEBlock(L, torch.ones(512, device="cuda"), torch.zeros(512, device="cuda"))
    x = torch.zeros(8, 512, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        blk.decode(x)
        g = torch.cuda.CUDAGraph()
        st.synchronize()
        with torch.cuda.graph(g, stream=st):
            out = blk.decode(x)
    x.copy_(wl.x[0].torch("cuda"))
    torch.cuda.synchronize()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    check_no_device_error()
    assert torch.equal(out, layer.MoEBlock(L, blk.gamma, blk.beta).decode(x))
