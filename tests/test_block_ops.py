"""Operators around the layer, host side: refusals, sizes, and the tests' own 64-bit forms."""
import ctypes

import numpy as np
import pytest

import _block_ref as ref
import routing_permute_grouped_router_gb300 as pkg
from routing_permute_grouped_router_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pkg.lib()


def status(rc):
    return pkg.STATUS[rc]


A = 0x10000  # an aligned address; nothing here gets as far as using it


def test_philox_known_answers():
    """The generator's published test vectors."""
    def words(*w):
        return [np.array([v], np.uint64) for v in w]

    assert [int(v[0]) for v in ref.philox(words(0, 0, 0, 0), [0, 0])] == \
        [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert [int(v[0]) for v in ref.philox(words(f, f, f, f), [f, f])] == \
        [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_norm_formula_against_differences():
    rng = np.random.default_rng(3)
    x, dy, u = (rng.standard_normal((5, 37)) for _ in range(3))
    gamma, beta, ug = 1 + 0.2 * rng.standard_normal(37), rng.standard_normal(37), rng.standard_normal(37)
    _, mean, rstd = ref.norm_fwd(x, gamma, beta, 1e-5)
    dx, dgamma, dbeta = ref.norm_bwd(x, dy, gamma, mean, rstd)

    def loss(s, sg):
        return (ref.norm_fwd(x + s * u, gamma + sg * ug, beta + sg * ug, 1e-5)[0] * dy).sum()

    e = 1e-5
    assert abs((loss(e, 0) - loss(-e, 0)) / (2 * e) - (dx * u).sum()) < 1e-6
    assert abs((loss(0, e) - loss(0, -e)) / (2 * e) - ((dgamma + dbeta) * ug).sum()) < 1e-6


@pytest.mark.parametrize("kw,err", [
    (dict(T=65), "MOE_ERR_SHAPE"), (dict(T=-1), "MOE_ERR_SHAPE"), (dict(d_model=100), "MOE_ERR_SHAPE"),
    (dict(k=9, E=16), "MOE_ERR_SHAPE"), (dict(E=129), "MOE_ERR_SHAPE"), (dict(dtype=5), "MOE_ERR_DTYPE"),
])
def test_decode_refuses_configs(lib, kw, err):
    cfg = pkg.config(**{**dict(T=8, d_model=256, d_ff=256, E=4, k=2), **kw})
    with pytest.raises(pkg.MoeError, match=err):
        pkg.moe_decode_workspace_size(cfg)
    w = pkg.MoeWeights(A, None, A, A, A)
    assert status(lib.moe_layer_decode(ctypes.byref(cfg), ctypes.byref(w), A, None, A, None, None, A, 1 << 40,
                                       None)) == err


def test_decode_refuses_pointers(lib):
    cfg = pkg.config(8, 256, 256, 4, 2)
    size = pkg.moe_decode_workspace_size(cfg)
    assert size >= 8 * 2 * 256 * 4

    def call(w=(A, None, A, A, A), x=A, res=None, y=A, ids=None, gates=None, ws=A, n=size, c=cfg):
        weights = pkg.MoeWeights(*w)
        return status(lib.moe_layer_decode(ctypes.byref(c), ctypes.byref(weights), x, res, y, ids, gates, ws, n, None))

    n0 = lib.moe_launch_count()
    assert call(x=None) == "MOE_ERR_INVALID_ARG"
    assert call(y=None) == "MOE_ERR_INVALID_ARG"
    assert call(x=A + 2) == "MOE_ERR_ALIGNMENT"
    assert call(res=A + 8) == "MOE_ERR_ALIGNMENT"
    assert call(ids=A + 1) == "MOE_ERR_ALIGNMENT"
    assert call(w=(None, None, A, A, A)) == "MOE_ERR_INVALID_ARG"
    assert call(w=(A, None, A, A + 4, A)) == "MOE_ERR_ALIGNMENT"
    assert call(ws=None) == "MOE_ERR_WORKSPACE"
    assert call(n=size - 1) == "MOE_ERR_WORKSPACE"
    assert status(lib.moe_layer_decode(ctypes.byref(cfg), None, A, None, A, None, None, A, size, None)) == \
        "MOE_ERR_INVALID_ARG"
    assert lib.moe_launch_count() == n0


def test_norm_refusals(lib):
    def fwd(rows=4, d=64, dtype=1, x=A, gamma=A, beta=A, eps=1e-5, y=A, mean=A, rstd=A):
        return status(lib.moe_norm_fwd(rows, d, dtype, x, gamma, beta, eps, y, mean, rstd, None))

    def bwd(rows=4, d=64, dtype=1, x=A, dy=A, gamma=A, mean=A, rstd=A, res=None, dx=A, dg=A, db=A, acc=0, ws=A,
            n=1 << 30):
        return status(lib.moe_norm_bwd(rows, d, dtype, x, dy, gamma, mean, rstd, res, dx, dg, db, acc, ws, n, None))

    n0 = lib.moe_launch_count()
    for f in (fwd, bwd):
        assert f(rows=-1) == "MOE_ERR_SHAPE"
        assert f(d=0) == "MOE_ERR_SHAPE"
        assert f(d=65537) == "MOE_ERR_SHAPE"
        assert f(rows=1 << 40) == "MOE_ERR_SHAPE"
        assert f(dtype=2) == "MOE_ERR_DTYPE"
        assert f(x=None) == "MOE_ERR_INVALID_ARG"
        assert f(x=A + 4) == "MOE_ERR_ALIGNMENT"
        assert f(gamma=None) == "MOE_ERR_INVALID_ARG"
        assert f(mean=A + 2) == "MOE_ERR_ALIGNMENT"
    for eps in (-1e-5, float("nan"), float("inf")):
        assert fwd(eps=eps) == "MOE_ERR_INVALID_ARG"
    assert bwd(acc=2) == "MOE_ERR_INVALID_ARG"
    assert bwd(mean=None) == "MOE_ERR_INVALID_ARG"
    assert bwd(dg=None) == "MOE_ERR_INVALID_ARG"
    assert bwd(res=A + 8) == "MOE_ERR_ALIGNMENT"
    assert bwd(ws=None) == "MOE_ERR_WORKSPACE"
    assert bwd(n=pkg.moe_norm_workspace_size(4, 64) - 1) == "MOE_ERR_WORKSPACE"
    assert lib.moe_launch_count() == n0


def test_dropout_refusals(lib):
    def add(n=8, dtype=1, y=A, res=None, out=A, p=0.1):
        return status(lib.moe_dropout_add(n, dtype, y, res, out, p, 1, 2, None))

    def bwd(n=8, dtype=1, y=A, out=A, p=0.1):
        return status(lib.moe_dropout_bwd(n, dtype, y, out, p, 1, 2, None))

    n0 = lib.moe_launch_count()
    for f in (add, bwd):
        for p in (-0.1, 1.0, 1.5, float("nan"), float("inf"), 1 - 2.0 ** -18):  # the last rounds to 1
            assert f(p=p) == "MOE_ERR_INVALID_ARG"
        assert f(n=-1) == "MOE_ERR_SHAPE"
        assert f(n=(1 << 40) + 1) == "MOE_ERR_SHAPE"
        assert f(dtype=3) == "MOE_ERR_DTYPE"
        assert f(y=None) == "MOE_ERR_INVALID_ARG"
        assert f(out=A + 2) == "MOE_ERR_ALIGNMENT"
    assert add(res=A + 4) == "MOE_ERR_ALIGNMENT"
    assert lib.moe_launch_count() == n0


def test_binding_refuses_mismatched_tensors(lib):
    import torch

    x, v = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError):  # tensors on the CPU
        pkg.moe_norm_fwd(x, v, v, 1e-5, x)
    with pytest.raises(TypeError):
        pkg.moe_dropout_add(x.half(), None, x.half(), 0.1, 0, 0)
    f32 = torch.float32
    with pytest.raises(TypeError):
        pkg._arg("y", x.bfloat16(), 32, f32)
    with pytest.raises(ValueError):
        pkg._arg("y", x[:2], 32, f32)
    with pytest.raises(ValueError):
        pkg._arg("gamma", v, 9, f32)
    with pytest.raises(ValueError):
        pkg._arg("y", x.t(), 32, f32)
    assert pkg._arg("residual", None, 32, f32) is None
    cfg = pkg.config(4, 8, 8, 2, 1, dtype=pkg.MOE_F32)
    with pytest.raises(TypeError):
        pkg.moe_layer_decode(cfg, {}, x.bfloat16(), None, x, None, None, x)
