"""The bounds that the float32 vocabulary loss is tested against tell a product of parts that is missing (host only)."""
import pytest
import torch

import _loss_bits as bits
import _step_ref as ref

PAIRS = [(i, j) for i in range(3) for j in range(3 - i)]


@pytest.mark.parametrize("T", [40, 300])
def test_forward_bound_tells_a_missing_product(T):
    x, W, labels, exact = bits.forward_case(T, 1000, 512, T)
    _, lse, _ = ref.loss_fwd(x, W, labels)
    assert (lse - exact).abs().max() <= 2.0 ** -40  # the other words are too far below
    at = x.argmax(1)
    a, b = bits.parts(x[torch.arange(T), at]), bits.parts(W[:, at].max(0).values)
    off = lambda z: float(((z - exact).abs() / exact).max())  # noqa: E731
    assert off(bits.product(a, b)) <= 8 * bits.U
    assert all(off(bits.product(a, b, p)) > 3 * bits.FORWARD for p in PAIRS)


@pytest.mark.parametrize("T,token", [(5, None), (300, None), (5, 0), (300, 299)])
def test_backward_bound_tells_a_missing_product(T, token):
    x, W, labels, lse, dloss = bits.backward_case(T, 264, 300, T, 150, token)
    dx, dW, dz, _ = ref.loss_bwd(x, W, labels, lse, dloss)
    dz = dz[:, 150]
    others = dx - dz[:, None] * W[150].double()
    assert others.abs().max() <= 1e-15  # the other words hold nothing
    for exact, left, right in ((dx, dz[:, None], W[150][None]),) + (((dW[150][None], dz[token, None, None], x[token][None]),) if token is not None else ()):
        a, b = bits.parts(left.float(), True), bits.parts(right)
        off = lambda v: float(((v - exact).abs() / exact.abs()).max())  # noqa: E731
        assert off(bits.product(a, b)) <= 5 * bits.U  # dz is a float32 here
        assert all(off(bits.product(a, b, p)) > 3 * bits.BACKWARD for p in PAIRS)
