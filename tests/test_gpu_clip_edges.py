"""Gradient clipping: what its order of summation depends on, and scales that are no normal float32."""
import pytest
import torch

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


def clipped(src, dst, max_norm):
    norm = torch.full((1,), float("nan"), device="cuda")
    pkg.moe_clip_grads(pkg.grad_list(src, dst), max_norm, norm, pkg.clip_workspace(len(src)).fill_(255))
    return norm


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_clip_repeats_itself_at_the_same_place_modulo_16_bytes(dtype):
    """Copies of the gradients elsewhere, each as far past a multiple of 16 bytes as before: the same bits."""
    t = ops.TYPES[dtype]
    unit = 16 // torch.empty(0, dtype=t).element_size()
    sizes = (8192, 16384, 70001, 5, 300007)
    values = [ops.rand(n, seed=n, dtype=t, scale=3.0 ** (i - 2)) for i, n in enumerate(sizes)]
    for first in range(unit):
        results = []
        for shift in (0, unit, 37 * unit):
            flat = torch.zeros(sum(sizes) + 64 * unit * len(sizes), dtype=t, device="cuda")
            src, at = [], shift + first
            for i, v in enumerate(values):
                flat[at:at + v.numel()] = v
                src.append(flat[at:at + v.numel()])
                at += v.numel() + (shift + unit) * (i % 3)  # and other distances between them
                at += (first + 3 * i - at) % unit
            dst = [torch.empty_like(v) for v in values]
            results.append((clipped(src, dst, 0.5 * ops.norm64(values)), *dst))
        for r in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], r)), first
    check_no_device_error()
