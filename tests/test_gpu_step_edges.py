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
