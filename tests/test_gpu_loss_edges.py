"""The vocabulary loss where its values are infinite, and how many of its bits are right."""
import math

import pytest
import torch

import _loss_bits as bits
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


@pytest.mark.parametrize("T", [1, 4, 20, 64, 65, 300])
@pytest.mark.parametrize("words", [(7,), (7, 9), (7, 399), (3, 130, 260, 399)])
def test_loss_of_infinite_logits(T, words):
    """lse is inf, as log sum exp is; the loss of any other label is inf, that of such a word has no value."""
    x, W, labels = ops.loss_inputs(T, 72, 400, torch.bfloat16, seed=T)
    x = x.abs() + 0.01
    W[words, :] = float("inf")
    W[50:60] = float("-inf")
    labels = (labels % 100 + 270).int()
    labels[::3] = words[0]
    labels[1::5] = 55
    labels[2::7] = -100
    loss, lse, _ = ops.run_loss(x, W, labels)
    valid = labels >= 0
    at_word = labels == words[0]
    assert (lse[valid] == math.inf).all() and (lse[~valid] == 0).all() and (loss[~valid] == 0).all()
    assert loss[at_word].isnan().all() and (loss[valid & ~at_word] == math.inf).all()
    check_no_device_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [4, 40, 64, 130])
def test_loss_of_a_logit_past_float32(dtype, T):
    """One token's logit of one word is 2^160: that token's lse and loss are inf, the others are as they were."""
    x, W, labels = ops.loss_inputs(T, 72, 400, ops.TYPES[dtype], seed=T)
    x[:, 0] = 0
    W[:, 0] = 0
    labels[labels == 7] = 8
    clean = ops.run_loss(x, W, labels)
    x[3, 0], W[7, 0] = 2.0 ** 60, 2.0 ** 100
    loss, lse, _ = ops.run_loss(x, W, labels)
    rest = [i for i in range(T) if i != 3]
    assert lse[3] == math.inf and loss[3] == math.inf
    assert torch.equal(loss[rest], clean[0][rest]) and torch.equal(lse[rest], clean[1][rest])
    e_loss, e_lse, _ = ref.loss_fwd(x, W, labels)
    assert float(e_lse[3]) == 2.0 ** 160 and float(e_loss[3]) == 2.0 ** 160  # 64 bits hold it
    check_no_device_error()


@pytest.mark.parametrize("T,d", [(1, 1000), (8, 1000), (40, 1000), (48, 4096), (49, 1000), (300, 1000), (700, 260)])
def test_float32_loss_has_all_products(T, d):
    x, W, labels, exact = bits.forward_case(T, d, 512, T)
    loss, lse, _ = ops.run_loss(x.cuda(), W.cuda(), labels.cuda())
    e_loss, _, _ = ref.loss_fwd(x, W, labels)
    assert ((lse.cpu().double() - exact).abs() <= bits.FORWARD * exact).all()
    assert ((loss.cpu().double() - e_loss).abs() <= bits.FORWARD * (exact + (exact - e_loss).abs())).all()
    check_no_device_error()


@pytest.mark.parametrize("T,token", [(1, None), (5, None), (300, None), (700, None), (1, 0), (5, 3), (300, 0), (300, 150), (300, 299), (700, 600)])
@pytest.mark.parametrize("word", [0, 150, 299])
def test_float32_gradients_have_all_products(T, token, word):
    x, W, labels, lse, dloss = (v.cuda() for v in bits.backward_case(T, 264, 300, T + word, word, token))
    dx, dW = ops.run_loss_bwd(x, W, labels, lse, dloss, torch.float32)
    e_dx, e_dW, _, _ = ref.loss_bwd(x, W, labels, lse, dloss)
    assert ((dx.double() - e_dx).abs() <= bits.BACKWARD * e_dx.abs()).all()
    if token is not None or T == 1:
        assert ((dW[word].double() - e_dW[word]).abs() <= bits.BACKWARD * e_dW[word].abs()).all()
    check_no_device_error()


@pytest.mark.parametrize("T,d,V", [(1, 16384, 1000), (60, 4096, 1000), (300, 1024, 5003), (1000, 64, 300001), (1000, 512, 1000)])
@pytest.mark.parametrize("dw", [None, torch.bfloat16, torch.float32])
def test_dx_has_the_label_term_beyond_8_bits(T, d, V, dw):
    """Logits of nearly 0 and a dz of each label that is nearly halfway between two bf16 values: its rounding would be 0.35 %
    of all of dx.  dx's own roundings are at random, so along the exact dx next to nothing of them is left."""
    W = ops.rand(V, d, seed=T + V, dtype=torch.bfloat16)
    x = (ops.rand(T, d, seed=T) * 2.0 ** -60).bfloat16()
    labels = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(T)).int().cuda()
    labels[0] = V - 1
    lse = torch.full((T,), float(V), device="cuda").log()
    p = torch.exp(-lse[0].double())
    dloss = torch.full((T,), float((1 + 0.9 * 2.0 ** -8) / (1 - p)), device="cuda") * 2.0 ** torch.arange(T, device="cuda").remainder(5)
    off = float((dloss.double() * (1 - p) / (dloss.double() * (1 - p)).bfloat16().double() - 1).abs().min())
    assert off > 0.8 * 2.0 ** -8
    dx, _ = ops.run_loss_bwd(x, W, labels, lse, dloss, dw, dW=dw is not None)
    g = dloss.double()[:, None]
    spread = g * p * W.double().sum(0)  # of all words; they share p and so the rounding of g p
    exact = spread - g * W[labels.long()].double()
    n = exact.square().sum()
    along = float(((dx.double() - exact) * exact).sum() / n)
    # half a step of bf16 on each element, of independent sign: seven times the root of the sum of their squares
    own = 7 * 2.0 ** -8 * float(exact.pow(4).sum().sqrt() / n)
    words = 2.0 ** -8 * float((spread * exact).sum().abs() / n)
    assert own + words < 0.5 * off, "the case does not tell the term"
    assert abs(along) <= own + words + 2.0 ** -20, f"{along:.2e} along dx, {own + words:.2e} at most"
    check_no_device_error()


@pytest.mark.parametrize("T", [1, 16, 33, 64])
@pytest.mark.parametrize("at", [0, 130, 1024, 2500, 4095])
def test_logits_of_few_bf16_tokens_lose_little_beside_a_large_product(T, at):
    """One word, so lse is its logit: a product of 2^24, at `at`, and 4095 of 1/32.

    The tensor core cuts a sum off, so what 16 small products give, 1/2, is lost on top of the large one, whose steps are
    2 (or 1, with a bit more).  That ends with the sum over K = 256 that has it: 16 halves at most.  The others are 8
    each, exact, and so are their sums with it, but for one rounding by at most 1.  (32 would be lost of a K of 1024.)
    """
    x, W = torch.full((T, 4096), 1 / 32, device="cuda"), torch.ones(1, 4096, device="cuda")
    x[:, at], W[:, at] = 4096, 4096
    _, lse, _ = ops.run_loss(x.bfloat16(), W.bfloat16(), torch.zeros(T, dtype=torch.int32, device="cuda"))
    lost = 2.0 ** 24 + 4095 / 32 - lse.double()
    assert -1 <= float(lost.min()) and float(lost.max()) <= 9, f"{float(lost.max())} lost"
    check_no_device_error()


@pytest.mark.parametrize("T", [49, 300])
@pytest.mark.parametrize("at", [0, 130, 1024, 2500, 4095])
def test_logits_of_float32_tokens_lose_little_beside_a_large_product(T, at):
    """The same in float32, on the tensor cores from 49 tokens on: 32 halves of the sum over K = 512 that has it."""
    x, W = torch.full((T, 4096), 1 / 32, device="cuda"), torch.ones(1, 4096, device="cuda")
    x[:, at], W[:, at] = 4096, 4096
    _, lse, _ = ops.run_loss(x, W, torch.zeros(T, dtype=torch.int32, device="cuda"))
    lost = 2.0 ** 24 + 4095 / 32 - lse.double()
    assert -1 <= float(lost.min()) and float(lost.max()) <= 17, f"{float(lost.max())} lost"
    check_no_device_error()
