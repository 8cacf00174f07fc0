"""Paths of the operators around the layer that a call takes only at some sizes, against their 64-bit forms.

The tolerances are those of test_gpu_block_ops, whose helpers are used here.
"""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import _block_ref as ref
import routing_permute_grouped_router_gb300 as pkg
from _util import check_no_device_error, to64
from routing_permute_grouped_router_gb300 import layer
from routing_permute_grouped_router_gb300 import workload as W
from test_gpu_block_ops import TYPES, check_decode, decode, decode_ref, near, norm_inputs

pytestmark = pytest.mark.gpu
LS = W.LayerShape


@pytest.fixture(scope="module", autouse=True)
def built():
    from routing_permute_grouped_router_gb300 import build

    build.build()
    pkg.lib()
    torch.cuda.set_device(0)
    pkg.moe_get_device_error(clear=True)


# ----------------------------- few-token layer, bf16 ----------------------- #
def up_product_split(shape, ids, ctas):
    """(few rows, units of a CTA, tiles in one CTA, tiles in several) of one half of the up product of a dropless
    bf16 call: units of 64 rows of d, tiles of 128 columns of f, split evenly over the CTAs."""
    nact, rows = len(np.unique(ids)), ids.size
    per_tile, tiles = shape.d_model // 64, nact * (shape.d_ff // 256)
    base, more = divmod(per_tile * tiles, ctas)
    begin = [c * base + min(c, more) for c in range(ctas + 1)]
    owner = np.searchsorted(begin, np.arange(per_tile * tiles), side="right") - 1
    owner = owner.reshape(tiles, per_tile)
    whole = int((owner[:, 0] == owner[:, -1]).sum())
    return rows <= 64 and rows <= 2 * nact, base, whole, tiles - whole


FEW_ROWS = [
    LS("top8_e64", 8, 256, 1024, 64, 8, 0.0, W.BF16),
    LS("one_token_long_f", 1, 256, 8192, 8, 8, 0.0, W.BF16),
    LS("two_tokens_long_d", 2, 4096, 1024, 8, 4, 0.0, W.BF16),
]


@pytest.mark.parametrize("shape", FEW_ROWS, ids=lambda s: s.name)
def test_decode_few_rows_with_whole_and_split_tiles(shape):
    """Calls with few rows make h from the up product's sums, whose tiles lie in one CTA or in several; again and
    again, since another CTA's sums must never be read before they are there."""
    wl = W.make(shape, seed=17, micro_batches=1, with_dy=False)
    e = decode_ref(wl, shape.T)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    few, _, whole, split = up_product_split(shape, e["ids"], sms)
    assert few and split > 0 and (whole > 0 or shape.d_model == 4096)
    r = decode(wl, shape.T)
    check_decode(r, e)
    first = r["y"].clone()
    for _ in range(50):
        r["ws"].fill_(255)
        pkg.moe_layer_decode(r["cfg"], r["w"], r["x"], None, r["y"], r["ids"], r["gates"], r["ws"])
        assert torch.equal(first, r["y"])
    check_no_device_error()


@pytest.mark.parametrize("shape", [LS("long_d", 64, 4096, 1536, 4, 4, 0.0, W.BF16),
                                   LS("one_row_each", 3, 4096, 1536, 8, 4, 0.0, W.BF16)], ids=lambda s: s.name)
def test_decode_many_units_a_cta(shape):
    """A CTA's share of the weights is longer than its ring of stages, whose places are used again."""
    wl = W.make(shape, seed=18, micro_batches=1, with_dy=False)
    e = decode_ref(wl, shape.T)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert up_product_split(shape, e["ids"], sms)[1] >= 10  # of at most eight stages
    check_decode(decode(wl, shape.T), e)


# ----------------------------- several rows to a group of threads ---------- #
LONG = [(3001, 4096), (1500, 8192), (12001, 1021), (24001, 60), (24001, 129), (2000, 10001), (1300, 16384)]


def near_sum(name, got, exp, terms, rel=0.0, size=None):
    """Sums of `terms` comparable fp32 terms: sqrt(terms) roundings, 64 at least, of the largest value (or `size`)."""
    big = 2.0 ** -24 * max(64.0, terms ** 0.5)
    scale = 1.0 if size is None else max(1.0, size / max(np.abs(exp).max(), 1e-30))
    near(name, got, exp, rel, big * scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", LONG)
def test_norm_of_many_rows(rows, d, dtype):
    """Every group of threads takes several rows, more than its ring has places where the ring is used."""
    x, dy, res, gamma, beta = norm_inputs(rows, d, dtype, seed=rows + d)
    f = dict(dtype=torch.float32, device="cuda")
    y, mean, rstd = torch.full_like(x, float("nan")), torch.empty(rows, **f), torch.empty(rows, **f)
    pkg.moe_norm_fwd(x, gamma, beta, 1e-5, y, mean, rstd)
    x64, dy64, g64 = to64(x), to64(dy), to64(gamma)
    ey, emean, erstd = ref.norm_fwd(x64, g64, to64(beta), 1e-5)
    near_sum("y", y, ey, d)
    near_sum("mean", mean, emean, d)
    near_sum("rstd", rstd, erstd, d)

    m64, r64 = to64(mean), to64(rstd)
    edx, edg, edb = ref.norm_bwd(x64, dy64, g64, m64, r64)
    size = np.abs(r64[:, None] * dy64 * g64).max()  # of the terms of dx
    ws = pkg.norm_workspace(rows, d).fill_(255)
    dg, db = torch.full((d,), 3.0, device="cuda"), torch.full((d,), -2.0, device="cuda")
    dx = torch.full_like(x, float("nan"))
    pkg.moe_norm_bwd(x, dy, gamma, mean, rstd, None, dx, dg, db, False, ws)
    near_sum("dx", dx, edx, d, size=size)
    near_sum("dgamma", dg, edg, rows)
    near_sum("dbeta", db, edb, rows)
    pkg.moe_norm_bwd(x, dy, gamma, mean, rstd, res, dx, dg, db, True, ws)
    near_sum("dx + dres", dx, edx + to64(res), d, size=size)
    near_sum("2 dgamma", dg, 2 * edg, rows)
    near_sum("2 dbeta", db, 2 * edb, rows)

    # in place of each input: the same bits
    pkg.moe_norm_bwd(x, dy, gamma, mean, rstd, res, dx, dg, db, False, ws)
    want = [t.clone() for t in (dx, dg, db)]
    for i in range(3):
        t = [x.clone(), dy.clone(), res.clone()]
        pkg.moe_norm_bwd(t[0], t[1], gamma, mean, rstd, t[2], t[i], dg, db, False, ws)
        assert torch.equal(t[i], want[0]) and torch.equal(dg, want[1]) and torch.equal(db, want[2])
    z = x.clone()
    pkg.moe_norm_fwd(z, gamma, beta, 1e-5, z)
    assert torch.equal(z, y)
    check_no_device_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropout_of_many_blocks(dtype):
    """Every thread takes several blocks of eight, the next loaded while this one is drawn for."""
    n, p, seed, offset = (1 << 23) + 5, 0.3, 0x123456789ABCDEF, 77
    y, r = (torch.randn(n, device="cuda").to(TYPES[dtype]) for _ in range(2))
    y[y == 0] = 1
    e = ref.dropout(to64(y), p, seed, offset)
    out = torch.full_like(y, float("nan"))
    pkg.moe_dropout_add(y, None, out, p, seed, offset)
    assert np.array_equal(to64(out) != 0, e != 0)
    near("out", out, e, rel=2.0 ** -22, big=0)
    dy = torch.empty_like(y)
    pkg.moe_dropout_bwd(y, dy, p, seed, offset)
    assert torch.equal(out, dy)
    pkg.moe_dropout_add(y, r, out, p, seed, offset)
    near("out + residual", out, e + to64(r), rel=2.0 ** -22, big=2.0 ** -22)
    kept = torch.from_numpy(e != 0).cuda()
    assert torch.equal(out[~kept], r[~kept])
    z = r.clone()
    pkg.moe_dropout_add(y, z, z, p, seed, offset)
    assert torch.equal(z, out)
    check_no_device_error()


# ----------------------------- the block's buffers ------------------------- #
def serving_block():
    wl = W.make(LS("serve", 64, 512, 256, 8, 2, 0.0, W.BF16), seed=23, micro_batches=1, with_dy=False)
    L = layer.from_workload(wl, training=False)
    blk = layer.MoEBlock(L, torch.ones(512, device="cuda"), torch.zeros(512, device="cuda"))
    return blk, wl.x[0].torch("cuda"), lambda: layer.MoEBlock(L, blk.gamma, blk.beta)


def test_block_decode_graphs_of_several_sizes():
    """One graph a batch size, captured in ascending order, each replayed after the others were made and memory has
    been handed out again."""
    blk, x, fresh = serving_block()
    st = torch.cuda.Stream()
    sizes, graphs, xs, outs = (1, 8, 40, 64), [], [], []
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for T in sizes:
            xs.append(torch.zeros(T, 512, dtype=torch.bfloat16, device="cuda"))
            blk.decode(xs[-1])
            st.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=st):
                outs.append(blk.decode(xs[-1]))
    blk.decode(x)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    others = [torch.full((n << 20,), 255, dtype=torch.uint8, device="cuda") for n in (1, 2, 4, 8, 16, 32, 64) * 2]
    for seed in range(3):
        want = [fresh().decode(x[seed:seed + T].contiguous()).clone() if seed + T <= 64 else None for T in sizes]
        for T, g, xi, out, e in reversed(list(zip(sizes, graphs, xs, outs, want))):
            if e is not None:
                xi.copy_(x[seed:seed + T])
                g.replay()
                assert torch.equal(out, e)
    check_no_device_error()
    assert all(bool((o == 255).all()) for o in others)  # nothing was written into memory that others own


def test_block_decode_on_two_streams():
    blk, x, fresh = serving_block()
    want = [fresh().decode(x[i:i + 24].contiguous()).clone() for i in (0, 40)]
    xs = [x[i:i + 24].contiguous() for i in (0, 40)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [blk.decode(xi, stream=s) for xi, s in zip(xs, streams)]
    torch.cuda.synchronize()
    check_no_device_error()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_block_decode_after_refused_calls():
    blk, x, fresh = serving_block()
    want = fresh().decode(x[:4].contiguous())
    n0 = pkg.moe_launch_count()
    for bad, err in ((x[:4].float(), TypeError), (x[:4, :256].contiguous(), ValueError), (x[:4].cpu(), ValueError),
                     (torch.cat([x, x[:1]]), pkg.MoeError)):
        with pytest.raises(err):
            blk.decode(bad)
    assert pkg.moe_launch_count() == n0
    assert torch.equal(blk.decode(x[:4].contiguous()), want)
    check_no_device_error()


def test_block_of_no_tokens():
    """T = 0, as the layer takes it: empty results, zero gradients when overwriting, untouched when accumulating."""
    s = LS("empty", 0, 256, 256, 4, 2, 1.25, W.BF16, backward=True)
    L = layer.from_workload(W.make(s.replace(T=8), micro_batches=1, with_dy=True), T=0)
    blk = layer.MoEBlock(L, torch.ones(256, device="cuda"), torch.zeros(256, device="cuda"), p=0.1)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    grads = [blk.dgamma, blk.dbeta] + [L.grads[n] for n in ("dW_r", "dW1", "dW3", "dW2")]
    for g in grads:
        g.fill_(3.0)
    assert blk.forward(x, 1, 2).shape == blk.decode(x).shape == (0, 256)
    for accumulate, value in ((True, 3.0), (False, 0.0)):
        assert blk.backward(x, x, accumulate, 1, 2).shape == (0, 256)
        assert all(bool((g == value).all()) for g in grads)
    check_no_device_error()


# ----------------------------- calls from other threads -------------------- #
def test_calls_from_a_thread_that_has_used_nothing_yet():
    """A thread's first CUDA call may be the few-token layer or the grouped FFN, both of which begin with tensor maps."""
    wl = W.make(LS("thread", 8, 256, 256, 4, 2, 0.0, W.BF16), seed=24, micro_batches=1, with_dy=False)
    e = decode_ref(wl, 8)
    r = decode(wl, 8)
    L = layer.from_workload(wl)
    L.forward(r["x"])
    torch.cuda.synchronize()
    sv, w, failed = L.saved, r["w"], []
    y_perm = sv["y_perm"].clone()
    r["y"].fill_(float("nan"))
    stream = torch.cuda.current_stream()

    def few():
        pkg.moe_layer_decode(r["cfg"], w, r["x"], None, r["y"], r["ids"], r["gates"], r["ws"], stream)

    def ffn():
        pkg.moe_grouped_ffn(L.cfg, sv["x_perm"], sv["counts"], sv["offsets"], w["W1"], w["W3"], w["W2"], sv["h"],
                            sv["y_perm"], sv["a"], sv["b"], stream)

    def guarded(call):
        try:
            call()
        except Exception as ex:
            failed.append(repr(ex))

    for call in (few, ffn):
        t = threading.Thread(target=guarded, args=(call,))
        t.start()
        t.join()
    assert not failed, failed
    check_decode(r, e)
    assert torch.equal(y_perm.view(torch.int16), sv["y_perm"].view(torch.int16))


FIRST_CALLS = '''
import sys, threading
import torch
import routing_permute_grouped_router_gb300 as pkg
from routing_permute_grouped_router_gb300 import layer, workload as W

torch.cuda.set_device(0)
wl = W.make(W.LayerShape("first", 256, 256, 256, 8, 2, 0.0, W.BF16, backward=True), seed=1, micro_batches=1, with_dy=True)
x, dy = wl.x[0].torch("cuda"), wl.dy[0].torch("cuda")
layers = [layer.from_workload(wl) for _ in range(8)]
cfg = pkg.config(8, 256, 256, 8, 2)
few = [(torch.empty_like(x[:8]), pkg.decode_workspace(cfg)) for _ in layers]
torch.cuda.synchronize()
start, failed = threading.Barrier(len(layers)), []

def calls(i):
    try:
        v = torch.zeros(8, device="cuda")
        pkg.moe_norm_fwd(v, v, v, 1e-5, v)  # the thread's context and the error word
        start.wait()
        if sys.argv[1] == "few":
            pkg.moe_layer_decode(cfg, layers[i].weights, x[:8], None, few[i][0], None, None, few[i][1])
        else:
            layers[i].forward(x)
            layers[i].backward(x, dy, False)
    except Exception as e:
        failed.append(repr(e))

threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(layers))]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not failed, failed
assert pkg.moe_get_device_error() == (0, 0)
for i in range(1, len(layers)):
    assert torch.equal(few[0][0], few[i][0]) if sys.argv[1] == "few" else torch.equal(layers[0].y, layers[i].y)
'''


@pytest.mark.parametrize("kind", ["few", "layer"])
def test_first_calls_from_several_threads(kind):
    """Threads whose first calls of a process coincide all get the driver's tensor-map encoder."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS, kind], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
