"""A reorder that finds too few free pages leaves everything as it was, also over a table that names pages of count 0."""
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from test_gpu_reorder import i32, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("width", [4, 12000])  # a table that the CTA that plans rewrites, and one that it does not
def test_pages_that_were_given_back_already(width):
    cache, _, d_len, _ = make([13, 0, 0, 0, 17, 1], [0] * 6, 6, width=width)   # 2 + 3 + 1 pages: none is free
    row = cache.page_table[4, :3].tolist()
    cache.page_refs[row[0]] = 0                       # row 4: a page that nothing counts,
    cache.page_table[5, 0] = row[1]                   # one that row 5 names too though it is counted once,
    cache.page_table[4, 2] = 10 ** 6                  # and one that does not exist
    everything = (cache.page_table, cache.page_refs, d_len, cache.k, cache.v)
    before = [t.clone() for t in everything]
    # rows 4 and 5 leave two free pages, three are wanted
    assert int(cache.reorder(d_len, i32([0, 0, 0, 0, -1, -1]))) == 0
    assert sv.sv_query_status(cache.ws)[1] & sv.SV_DEV_OUT_OF_PAGES
    assert all(torch.equal(a, b) for a, b in zip(everything, before))
    # two are there; the pages given back too often are reported and left at 0 until they are taken
    assert int(cache.reorder(d_len, i32([0, 0, 0, -1, -1, -1]))) == 1
    assert sv.sv_query_status(cache.ws)[1] == sv.SV_DEV_BAD_PAGE
    first, last = before[0][0, :2].tolist()
    want = before[1].clone()
    want[first], want[last], want[row[0]], want[row[1]] = 3, 1, 1, 1
    assert torch.equal(cache.page_refs, want)
    low, high = sorted(row[:2])
    assert cache.page_table[:3, :2].tolist() == [[first, last], [first, low], [first, high]]
    assert (cache.page_table[3:] == -1).all() and d_len.tolist() == [13, 13, 13, 0, 0, 0]
