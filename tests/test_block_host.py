"""Host side of the block around the layer, without a GPU: its kernels' calls are recorded, not made."""
import contextlib
import weakref

import pytest
import torch

import routing_permute_grouped_router_gb300 as pkg
from routing_permute_grouped_router_gb300 import build as B
from routing_permute_grouped_router_gb300 import layer


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


@pytest.fixture
def block(monkeypatch):
    """(a block of a d = 256 layer on the CPU, the list of its few-token calls as (tokens, workspace, h, out))."""
    B.build()
    calls = []
    monkeypatch.setattr(layer, "moe_norm_fwd", lambda x, *a: None)
    monkeypatch.setattr(layer, "moe_layer_decode", lambda cfg, w, h, x, out, ids, gates, ws, stream: calls.append(
        (cfg.T, ws, h, out)))
    monkeypatch.setattr(layer.torch.cuda, "stream", lambda s: contextlib.nullcontext())

    class Layer:
        cfg = pkg.config(4, 256, 256, 4, 2)
        device, act_dtype, training, weights = torch.device("cpu"), torch.bfloat16, False, {}

    return layer.MoEBlock(Layer(), torch.ones(256), torch.zeros(256)), calls


def tokens(T, d=256):
    return torch.zeros(T, d, dtype=torch.bfloat16)


def test_decode_keeps_every_buffer_it_has_used(block):
    """A graph holds the addresses of the call that it captured: larger calls may not free them."""
    blk, calls = block
    s = Stream(7)
    for T in (1, 8, 64, 1, 8):
        blk.decode(tokens(T), s)
    kept = [[weakref.ref(t) for t in c[1:]] for c in calls]
    at = [[t.data_ptr() for t in c[1:]] for c in calls]
    sizes = [(c[0], c[1].numel()) for c in calls]
    calls.clear()
    assert all(r() is not None for c in kept for r in c)
    assert at[0] == at[3] and at[1] == at[4]
    for T, n in sizes:
        assert n >= pkg.moe_decode_workspace_size(pkg.config(T, 256, 256, 4, 2))


def test_decode_buffers_of_two_streams_are_apart(block):
    blk, calls = block
    for raw in (7, 9):
        blk.decode(tokens(8), Stream(raw))
        blk.decode(tokens(3), Stream(raw))
    ptrs = [{t.data_ptr() for t in c[1:]} for c in calls]
    assert not (ptrs[0] | ptrs[1]) & (ptrs[2] | ptrs[3])


def test_decode_after_a_refused_call(block, monkeypatch):
    """A call with a wrong type or width leaves no buffers of that type or width behind."""
    blk, calls = block
    s = Stream(7)

    def norm(x, gamma, beta, eps, y, *a):  # the binding's checks
        if y.dtype != x.dtype:
            raise TypeError
        if y.numel() != x.numel() or x.shape[-1] != gamma.numel():
            raise ValueError

    monkeypatch.setattr(layer, "moe_norm_fwd", norm)
    for x, err in ((tokens(4).float(), TypeError), (tokens(4, 128), ValueError), (tokens(65), pkg.MoeError)):
        with pytest.raises(err):
            blk.decode(x, s)
    assert not calls
    assert blk.decode(tokens(4), s).dtype == torch.bfloat16
    (T, ws, h, out), = calls
    assert h.shape == out.shape == (4, 256) and h.dtype == out.dtype == torch.bfloat16
    assert blk.decode(tokens(4).view(4, 1, 256), s).shape == (4, 1, 256)


def test_backward_without_training_buffers_says_so(block):
    blk, _ = block
    with pytest.raises(RuntimeError, match="without training buffers"):
        blk.backward(tokens(4), tokens(4), False)
