"""4-bit attention where one slot outweighs each of many others by 2^24 and more: their weights are small one by one, not together.
As many requests as leave every part of the line some whole contexts.

Bounds: a weight w enters the product with v as float16 under a reference at which the row's largest is 2^4 or more, so it is
off by at most half a step of the smallest float16, 2^-29 of the largest.  That times the slots, half a step of bf16 (2^-8), and
2^-10 of the value for scores of sums in float32, bound the difference."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from oracle import quant

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("D,heads", [(128, 1), (128, 8), (64, 16), (128, 20), (64, 40), (128, 64), (64, 100)])  # by rows; by tiles
@pytest.mark.parametrize("at", [0, 700, 1900])
@pytest.mark.parametrize("below", [24.0, 25.5, 27.0])
def test_many_small_weights(D, heads, at, below):
    B, n, page = 608, 2000, 64
    pages = -(-n // page)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = sv.PagedCache4.empty(1, pages, page, 1, D, B, pages)
    cache.reserve(i32([0]), i32([n]))
    k, v = torch.zeros((n, 1, D), device="cuda"), torch.ones((n, 1, D), device="cuda")
    k[at], v[at] = 1.0, 0.0
    cache.append(k.to(torch.bfloat16), v.to(torch.bfloat16), i32([0]), i32([0, n]))
    cache.page_table.copy_(cache.page_table[:1].expand(B, pages).contiguous())      # every request reads the same context
    q = torch.ones((B, heads, D), device="cuda").to(torch.bfloat16)
    pool = cache.pool[0].cpu().numpy()
    scale = below * np.log(2.0) / D / float(quant.read(pool, D, page, 1.0, False).max())
    out, lse = sv.tree_attention(q, cache, 0, i32([n - 1] * B), i32(list(range(B + 1))), None, 1, scale=scale)
    one, w = float(quant.read(pool, D, page, 1.0, True).max()), 2.0 ** -below
    want = one * (n - 1) * w / (1 + (n - 1) * w)
    assert np.abs(out.double().cpu().numpy() - want).max() <= n * 2.0 ** -29 + (2.0 ** -8 + 2.0 ** -10) * want
    assert np.abs(lse.double().cpu().numpy() - np.log(2.0 ** below + (n - 1))).max() <= D * 2.0 ** -24 * below + 2.0 ** -20
