"""Paths of the operators around the layer that a call takes only at some sizes, against their 64-bit forms.

The tolerances are those of test_gpu_block_ops, whose helpers are used here.
"""
import numpy as np
import pytest
import torch

import routing_permute_grouped_router_gb300 as pkg
from _util import check_no_device_error
from routing_permute_grouped_router_gb300 import workload as W
from test_gpu_block_ops import check_decode, decode, decode_ref

pytestmark = pytest.mark.gpu
LS = W.LayerShape


@pytest.fixture(scope="module", autouse=True)
def built():
    from routing_permute_grouped_router_gb300 import build

    build.build()
    pkg.lib()
    torch.cuda.set_device(0)
    pkg.moe_get_device_error(clear=True)


# ----------------------------- few-token layer, bf16 ----------------------- #
def up_product_split(shape, ids, ctas):
    """(few rows, units of a CTA, tiles in one CTA, tiles in several) of one half of the up product of a dropless
    bf16 call: units of 64 rows of d, tiles of 128 columns of f, split evenly over the CTAs."""
    nact, rows = len(np.unique(ids)), ids.size
    per_tile, tiles = shape.d_model // 64, nact * (shape.d_ff // 256)
    base, more = divmod(per_tile * tiles, ctas)
    begin = [c * base + min(c, more) for c in range(ctas + 1)]
    owner = np.searchsorted(begin, np.arange(per_tile * tiles), side="right") - 1
    owner = owner.reshape(tiles, per_tile)
    whole = int((owner[:, 0] == owner[:, -1]).sum())
    return rows <= 64 and rows <= 2 * nact, base, whole, tiles - whole


FEW_ROWS = [
    LS("top8_e64", 8, 256, 1024, 64, 8, 0.0, W.BF16),
    LS("one_token_long_f", 1, 256, 8192, 8, 8, 0.0, W.BF16),
    LS("two_tokens_long_d", 2, 4096, 1024, 8, 4, 0.0, W.BF16),
]


@pytest.mark.parametrize("shape", FEW_ROWS, ids=lambda s: s.name)
def test_decode_few_rows_with_whole_and_split_tiles(shape):
    """Calls with few rows make h from the up product's sums, whose tiles lie in one CTA or in several; again and
    again, since another CTA's sums must never be read before they are there."""
    wl = W.make(shape, seed=17, micro_batches=1, with_dy=False)
    e = decode_ref(wl, shape.T)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    few, _, whole, split = up_product_split(shape, e["ids"], sms)
    assert few and split > 0 and (whole > 0 or shape.d_model == 4096)
    r = decode(wl, shape.T)
    check_decode(r, e)
    first = r["y"].clone()
    for _ in range(50):
        r["ws"].fill_(255)
        pkg.moe_layer_decode(r["cfg"], r["w"], r["x"], None, r["y"], r["ids"], r["gates"], r["ws"])
        assert torch.equal(first, r["y"])
    check_no_device_error()
