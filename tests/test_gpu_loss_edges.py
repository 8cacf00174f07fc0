"""The vocabulary loss where its values are infinite, and how many of its bits are right."""
import math

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
