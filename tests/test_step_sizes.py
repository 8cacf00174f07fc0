"""Workspaces of the training step's operators serve smaller batches too (host only)."""
import pytest

import routing_permute_grouped_router_gb300 as pkg
from routing_permute_grouped_router_gb300 import build as B

F, H = pkg.MOE_F32, pkg.MOE_BF16


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def batches(upto):
    """Sizes of a batch around every border of a tile of tokens, and of the few."""
    near = {t + o for t in range(0, upto, 256) for o in (0, 1, 255)}
    return sorted(t for t in near | set(range(min(upto, 140))) if t <= upto)


# pieces of the vocabulary, slices of dx, the forms for few tokens, the smallest and the largest vocabularies and widths
@pytest.mark.parametrize("dtype", [H, F])
@pytest.mark.parametrize("d,V", [(8, 1), (64, 300), (64, 300001), (256, 1000), (2048, 50257), (4096, 65536), (4096, 128000), (65536, 100),
                                 (40000, 5000), (1000, 1 << 20)])
@pytest.mark.parametrize("training", [False, True])
def test_loss_workspace_serves_fewer_tokens(d, V, dtype, training):
    before = 0
    for T in batches(24000):
        size = pkg.moe_vocab_loss_workspace_size(T, d, V, dtype, training)
        assert size >= before, f"{T} tokens take {size} bytes, fewer {before}"
        assert not training or size >= pkg.moe_vocab_loss_workspace_size(T, d, V, dtype, False)
        before = size


@pytest.mark.parametrize("dtype", [H, F])
def test_loss_workspace_serves_fewer_of_very_many_tokens(dtype):
    """Past 2^20 tokens a piece is a tile's columns."""
    tokens = sorted([1 << e for e in range(25)] + [3 << e for e in range(23)] + [(1 << 24) - 1])
    sizes = [pkg.moe_vocab_loss_workspace_size(T, 64, 1 << 19, dtype, True) for T in tokens]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("d", [1, 31, 1021, 4096, 7001, 9001, 65536])
def test_row_workspaces_serve_fewer_rows(d):
    for size_of in (pkg.moe_residual_norm_workspace_size, pkg.moe_norm_workspace_size):
        sizes = [size_of(rows, d) for rows in (*range(0, 700), 1000, 1 << 14, 1 << 20)]
        assert sizes == sorted(sizes)


def test_clip_workspace_serves_fewer_tensors():
    sizes = [pkg.moe_clip_workspace_size(n) for n in (*range(0, 3000), 1 << 14, pkg.MOE_CLIP_MAX_TENSORS)]
    assert sizes == sorted(sizes)


def test_clip_overlaps_are_found_by_several_threads_at_once():
    """Lists of more tensors than the stack has room for share the library's: each call's answer is its own."""
    import ctypes
    import threading

    lib = pkg.lib()

    def entries(n, base, overlap):
        e = [pkg.MoeGrad(base + 64 * i, base + (1 << 30) + 64 * i, 16, F) for i in range(n)]
        if overlap is not None:
            e[overlap].dst += 4
        return (pkg.MoeGrad * n)(*e)

    def status(e, n):
        return pkg.STATUS[lib.moe_clip_grads(e, n, 1.0, ctypes.c_void_p(0x1000), 0x2000, 1 << 40, None)]

    sizes = (33, 40, 300, 2000)
    # what is refused here is refused before anything is launched; without a fault the call would go on, so none is made
    lists = [(entries(n, 1 << 34, n // 2), n) for n in sizes] + [(entries(n, 1 << 35, n - 2), n) for n in sizes]
    wrong = []

    def work():
        for _ in range(200):
            wrong.extend(n for e, n in lists if status(e, n) != "MOE_ERR_INVALID_ARG")

    threads = [threading.Thread(target=work) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
