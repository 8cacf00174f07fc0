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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top,most", [(2.0 ** 100, 2.0 ** -15), (2.0 ** 115, 2.0 ** -20), (2.0 ** 118, 2.0 ** -100), (2.0 ** 118, 2.0 ** -124),
                                      (2.0 ** 118, 2.0 ** -140), (2.0 ** 20, 2.0 ** -100), (2.0 ** 20, 2.0 ** -145), (2.0 ** -20, 2.0 ** -149)])
def test_clip_by_a_scale_that_is_no_normal_float32(dtype, top, most):
    """max_norm / norm is below 2^-126, or next to it: the clipped gradients have that norm all the same."""
    t = ops.TYPES[dtype]
    src = [(ops.rand(n, seed=n).double() * top).to(t) for n in (70001, 9)]
    src[0][5], src[1][3] = 0, -0.0
    total = ops.norm64(src)
    for dst in ([torch.full_like(v, float("nan")) for v in src], [v.clone() for v in src]):
        before = dst if dst[0].isnan().any() else None
        norm = clipped(src if before is not None else dst, dst, most)
        assert abs(float(norm) - total) <= ops.NORM * total
        for s, d in zip(src, dst):
            e = s.double() * (most / total)
            # the result's own rounding: half a step of the type, or of its smallest values; a bf16 one by way of float32
            room = (ops.NORM + 2 * ops.U + ops.HALF[t]) * e.abs() + (2.0 ** -134 if t == torch.bfloat16 else 0) + 2.0 ** -150
            assert ((d.double() - e).abs() <= room).all(), f"off by {float(((d.double() - e).abs() / room).max())} of the room"
    check_no_device_error()


def test_clip_of_long_lists_from_several_threads():
    """Each list is found sound and clipped as it is alone."""
    import threading

    lists = [[ops.rand(50 + i % 7, seed=1000 * k + i) for i in range(n)] for k, n in enumerate((33, 100, 300, 1000))]
    alone = []
    for src in lists:
        dst = [torch.empty_like(v) for v in src]
        alone.append((clipped(src, dst, 0.5), dst))
    torch.cuda.synchronize()
    failed = []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    dst = [torch.empty_like(v) for v in lists[k]]
                    norm = clipped(lists[k], dst, 0.5)
                    stream.synchronize()
                    assert torch.equal(norm, alone[k][0]) and all(torch.equal(a, b) for a, b in zip(dst, alone[k][1]))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k % 4,)) for k in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    check_no_device_error()
