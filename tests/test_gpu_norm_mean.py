"""The layer norm's mean: rows of one value, and rows whose mean is far larger than their deviation.

x - mean of a row of one value is 0.  The kernel's mean may be off by the rounding of its sum and of 1 / d, at most
26 roundings of 2^-24 of the value, but what the distances from it leave is taken off again, to a relative 2^-23: for
values up to 1000 and eps 1e-5 (1 / sqrt(eps) = 316) that leaves 6e-8 gamma of y, and y's own roundings 2^-24 beta each.
"""
import numpy as np
import pytest
import torch

import _block_ref as ref
import routing_permute_grouped_router_gb300 as pkg
from _util import check_no_device_error, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from routing_permute_grouped_router_gb300 import build

    build.build()
    pkg.lib()
    torch.cuda.set_device(0)
    pkg.moe_get_device_error(clear=True)


def run(x, gamma, beta):
    rows = x.shape[0]
    y, mean, rstd = torch.full_like(x, float("nan")), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    pkg.moe_norm_fwd(x, gamma, beta, 1e-5, y, mean, rstd)
    torch.cuda.synchronize()
    check_no_device_error()
    return y, mean, rstd


@pytest.mark.parametrize("d", [3, 100, 488, 1000, 1021, 4097, 5000, 8189, 10000, 10001, 65535])
def test_rows_of_one_value(d):
    values = [1000.0, 1.0, -7.0, 999.9, 1.0 / 3.0, 0.1, 0.0, 2.0 ** -20]
    x = torch.tensor(values, device="cuda")[:, None].expand(-1, d).contiguous()
    g = torch.Generator(device="cuda").manual_seed(d)
    gamma, beta = (torch.randn(d, generator=g, device="cuda") for _ in range(2))
    y, mean, rstd = run(x, gamma, beta)
    assert torch.equal(mean, x[:, 0])
    off = np.abs(to64(y) - to64(beta))
    assert (off <= 2.0 ** -23 * (np.abs(to64(gamma)) + np.abs(to64(beta)))).all()
    assert np.abs(to64(rstd) - 1e-5 ** -0.5).max() <= 2.0 ** -21 * 1e-5 ** -0.5  # rsqrtf: 2 ulp
    # in the backward x - mean is 0: dgamma is 0 and dx the projected dy
    dy = torch.randn(x.shape, generator=g, device="cuda")
    dx, dg, db = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    pkg.moe_norm_bwd(x, dy, gamma, mean, rstd, None, dx, dg, db, False, pkg.norm_workspace(len(values), d))
    assert not dg.any()


@pytest.mark.parametrize("d", [100, 1000, 4097, 10001])
def test_mean_far_larger_than_the_deviation(d):
    """x - mean is exact but for one rounding of what the distances leave: y is good to 32-bit roundings of the terms
    themselves, not of the mean."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x = 1000.0 + torch.randn(9, d, generator=g, device="cuda")
    gamma, beta = (torch.randn(d, generator=g, device="cuda") for _ in range(2))
    y, mean, rstd = run(x, gamma, beta)
    ey, emean, erstd = ref.norm_fwd(to64(x), to64(gamma), to64(beta), 1e-5)
    assert np.abs(to64(mean) - emean).max() <= 2.0 ** -23 * 1001  # two roundings, at the mean's size
    # sums of d comparable terms: sqrt(d) roundings, at most 64 here up to d = 4096 and 101 at 10001
    tol = 2.0 ** -24 * max(64, d ** 0.5)
    assert np.abs(to64(rstd) / erstd - 1).max() <= tol
    assert np.abs(to64(y) - ey).max() <= tol * np.abs(ey).max()


@pytest.mark.parametrize("d", [7, 64, 512, 1021, 4096, 4097, 8192])
@pytest.mark.parametrize("size", [30.0, 1000.0])
def test_one_channel_far_larger_than_the_others(d, size):
    """The first channel, which a sample of 32 elements (fewer in a short row) may hold: distances are then taken from
    a point `size` / 32 off, less than the deviation, size / sqrt(d), times sqrt(d) / 32.  What that point's square and
    the roundings at its size cost is (1 + d / 1024) and sqrt(d) / 32 times the usual."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(9, d, generator=g, device="cuda")
    x[:, 0] = size
    gamma, beta = (torch.randn(d, generator=g, device="cuda") for _ in range(2))
    y, mean, rstd = run(x, gamma, beta)
    ey, emean, erstd = ref.norm_fwd(to64(x), to64(gamma), to64(beta), 1e-5)
    ratio = 1 + max(d / 1024, 8)  # rows of up to 512 elements: samples of an eighth at least
    sums = 2.0 ** -24 * max(64, d ** 0.5)
    assert np.abs(to64(rstd) / erstd - 1).max() <= ratio * sums
    n = np.abs((ey - to64(beta)) / to64(gamma))
    tol = ratio * sums * n + 8 * 2.0 ** -24 * (n + 1 + d ** 0.5 / 32)
    assert (np.abs(to64(y) - ey) <= tol * np.abs(to64(gamma)) + 2.0 ** -23 * np.abs(to64(beta))).all()
    assert np.abs(to64(mean) - emean).max() <= sums * size
