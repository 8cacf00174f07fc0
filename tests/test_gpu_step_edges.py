"""The residual path between blocks where its kernels change: on either side of the longest rows that the ring in shared
memory takes, and rows that are not finite.  Tolerances are those of test_gpu_step_ops."""
import pytest
import torch

import _step_ref as ref
import routing_permute_grouped_router_gb300 as pkg
import test_gpu_step_ops as ops
from _util import check_no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from routing_permute_grouped_router_gb300 import build

    build.build()
    pkg.lib()
    torch.cuda.set_device(0)
    pkg.moe_get_device_error(clear=True)


# the backward's ring: float32 rows up to 5152 with four tensors and 6868 with three (without dout), 5121 and 6817
# where rows are no whole units, which take up to 127 bytes more; bf16 rows up to 8192 and 8185; 512 threads a row from 4097 on
@pytest.mark.parametrize("dtype,d,dout", [
    ("f32", 4100, True), ("f32", 4609, True), ("f32", 5120, True), ("f32", 5121, True), ("f32", 5122, True), ("f32", 5152, True),
    ("f32", 5156, True), ("f32", 6817, False), ("f32", 6818, False), ("f32", 6868, False), ("f32", 6872, False),
    ("f32", 8189, False), ("f32", 8190, False), ("bf16", 8185, True), ("bf16", 8186, True), ("bf16", 8192, True), ("bf16", 8193, True)])
@pytest.mark.parametrize("rows", [9, 310])
def test_join_on_either_side_of_the_ring(rows, d, dtype, dout):
    t = ops.TYPES[dtype]
    i = ops.join_inputs(rows, d, t, row=True, seed=d)
    r = ops.run_fwd(i, 0.8, 0.5)
    ops.check_fwd(r, ref.join_fwd(*i.values(), 0.8, 0.5))
    dh, do = ops.rand(rows, d, seed=8, dtype=t), ops.rand(rows, d, seed=9, dtype=t) if dout else None
    e = ref.join_bwd(r["out"], i["y"], dh, do, i["post"], i["nxt"], i["gate"], i["row"], 0.8, 0.5, r["ry"], r["ro"])
    b = ops.run_bwd(i, r, dh, do, 0.8, 0.5)
    ops.check_bwd(b, e)
    for dx, dy in ((0, 1), (1, 0)) if dout else ():  # in place
        given = [dh.clone(), do.clone()]
        c = ops.run_bwd(i, r, given[0], given[1], 0.8, 0.5, dx=given[dx], dy=given[dy])
        assert all(torch.equal(b[n], c[n]) for n in b)
    check_no_device_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [96, 512, 1021, 8192, 9000, 9001])
def test_join_rows_with_an_infinity(d, dtype):
    """An infinite x stays in out and gives ro = 0, so h is 0 but for a NaN in its place; an infinite y gives ry = 0, a NaN
    in its place of out and so a row of NaN in h.  The rows around them are as without them."""
    t = ops.TYPES[dtype]
    i = ops.join_inputs(20, d, t, seed=43)
    clean = ops.run_fwd(i)
    i["x"][6, 5], i["x"][7, d - 1], i["y"][11, 3] = float("inf"), float("-inf"), float("inf")
    r = ops.run_fwd(i)
    rest = [k for k in range(20) if k not in (6, 7, 11)]
    assert all(torch.equal(r[n][rest], clean[n][rest]) for n in r)
    for row, at, value in ((6, 5, float("inf")), (7, d - 1, float("-inf"))):
        others = [c for c in range(d) if c != at]
        assert r["out"][row, at] == value and torch.equal(r["out"][row, others], clean["out"][row, others])
        assert torch.equal(r["ry"][row], clean["ry"][row]) and r["ro"][row] == 0
        assert r["h"][row, at].isnan() and (r["h"][row, others] == 0).all()
    others = [c for c in range(d) if c != 3]
    assert r["ry"][11] == 0 and r["out"][11, 3].isnan() and torch.equal(r["out"][11, others], i["x"][11, others])
    assert r["ro"][11].isnan() and r["h"][11].isnan().all()
    check_no_device_error()
