"""The vocabulary loss on a workspace that was made for more tokens: its results, and nothing written behind it."""
import pytest
import torch

import routing_permute_grouped_router_gb300 as pkg
from _util import check_no_device_error

pytestmark = pytest.mark.gpu
BEHIND = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    from routing_permute_grouped_router_gb300 import build

    build.build()
    pkg.lib()
    torch.cuda.set_device(0)
    pkg.moe_get_device_error(clear=True)


def step(x, W, labels, ws, dw):
    T = x.shape[0]
    nan = lambda *s, t=torch.float32: torch.full(s, float("nan"), device="cuda", dtype=t)  # noqa: E731
    loss, lse, total, dx, dW = nan(T), nan(T), nan(2), nan(*x.shape, t=x.dtype), nan(*W.shape, t=dw)
    pkg.moe_vocab_loss_fwd(x, W, labels, loss, lse, ws, total)
    pkg.moe_vocab_loss_bwd(x, W, labels, lse, None, dx, dW, False, ws)
    return loss, lse, total, dx, dW


# 2^28 values of dz in one piece, two, three of the vocabulary; the forms for few tokens; dx in slices
@pytest.mark.parametrize("dtype,d,V,most,fewer", [
    ("bf16", 64, 300001, 1100, (1024, 900, 769, 768, 512, 257, 65, 64, 1)),
    ("bf16", 512, 100003, 2817, (2816, 2561, 2560, 300, 130)),
    ("f32", 64, 130003, 2100, (2049, 2048, 1025, 49, 48, 9, 1)),
    ("bf16", 8, 1, 500, (65, 64, 1)), ("f32", 132, 700, 600, (256, 100, 49, 48, 13))])
def test_loss_of_fewer_tokens_on_the_same_workspace(dtype, d, V, most, fewer):
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(most + V)
    x, W = (torch.randn(n, d, generator=g, device="cuda").to(t) for n in (most, V))
    labels = torch.randint(0, V, (most,), generator=g, device="cuda", dtype=torch.int32)
    labels[::7] = -100
    size = pkg.moe_vocab_loss_workspace_size(most, d, V, pkg.MOE_BF16 if t == torch.bfloat16 else pkg.MOE_F32, True)
    whole = torch.empty(size + BEHIND, dtype=torch.uint8, device="cuda")
    for dw in (torch.float32, torch.bfloat16) if t == torch.bfloat16 else (torch.float32,):
        for T in (most, *fewer):
            whole.fill_(165)
            a = step(x[:T], W, labels[:T], whole[:size], dw)
            own = torch.empty(pkg.moe_vocab_loss_workspace_size(T, d, V, pkg.MOE_BF16 if t == torch.bfloat16 else pkg.MOE_F32, True) + BEHIND,
                              dtype=torch.uint8, device="cuda").fill_(165)
            b = step(x[:T], W, labels[:T], own[:-BEHIND], dw)
            assert all(torch.equal(u, v) for u, v in zip(a, b)), T
            assert (whole[size:] == 165).all() and (own[-BEHIND:] == 165).all(), T
    check_no_device_error()
