"""The paged cache with rows that lack pages for their own length: a fork leaves them out and hands nothing out for them."""
import os
import sys

import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_cache import _gpu, i32, make, same  # noqa: E402, F401

pytestmark = pytest.mark.gpu
PS = 8


def filled(lens, rows, width, pages=400):
    """Rows 0..len(lens)-1 with pages for lens[i] slots, all others empty: (cache, oracle)."""
    cache, oracle = make(2, pages, PS, 2, 64, rows, width)
    full = list(lens) + [0] * (rows - len(lens))
    cache.reserve(i32([0] * rows), i32(full))
    oracle.reserve([0] * rows, full)
    same(cache, oracle)
    return cache, oracle


def hole(cache, oracle, row, entry, value=-1):
    """Entry `entry` of the row names `value` instead of its page, which becomes free."""
    oracle.refs[oracle.table[row, entry]] = 0
    oracle.table[row, entry] = value
    cache.page_refs.copy_(i32(oracle.refs))
    cache.page_table[row, entry] = value


# (length, entry that names no page): the last, partly filled page; a full one first, in the middle, last, past 32 entries
@pytest.mark.parametrize("n,entry", [(5, 0), (20, 2), (20, 0), (20, 1), (24, 2), (24, 1), (700, 87), (700, 86), (700, 40), (700, 31),
                                     (700, 32), (704, 87)])
@pytest.mark.parametrize("value", [-1, 400, 1 << 30, -7])
def test_fork_of_a_row_without_a_page(n, entry, value):
    rows, width = 6, 90
    cache, oracle = filled([n, 13, 16], rows, width)
    hole(cache, oracle, 0, entry, value)
    d = i32([n, 13, 16, 0, 0, 0])
    ok = cache.fork(d, i32([1, 0, 2]), i32([3, 4, 5]))
    lens = [n, 13, 16, 0, 0, 0]
    assert oracle.fork(MutableLens(lens), [1, 2], [3, 5]).tolist() == [1, 1]
    assert ok.tolist() == [1, 0, 1] and d.tolist() == [n, 13, 16, 13, 0, 16]
    assert sv.sv_query_status(cache.ws) == (sv.SV_ERR_DEVICE_INPUT, sv.SV_DEV_BAD_PAGE)
    same(cache, oracle)
    # the same without marks of the caller's
    cache.release(d, i32([3, 5]))
    oracle.release([0] * rows, [3, 5])
    sv.sv_cache_fork(cache.c, cache.page_table, width, rows, d, i32([0, 1]), i32([4, 3]), 2, None, cache.ws)
    oracle.fork(MutableLens(lens), [1], [3])
    assert d.tolist() == [n, 13, 16, 13, 0, 0] and sv.sv_query_status(cache.ws)[1] == sv.SV_DEV_BAD_PAGE
    same(cache, oracle)


class MutableLens(list):
    def copy(self):
        return MutableLens(self)


def test_a_missing_page_past_the_length_does_not_matter():
    cache, oracle = filled([24, 13], 4, 5)
    hole(cache, oracle, 0, 2)                 # slots 16 to 23, the row has 16 tokens
    d = i32([16, 13, 0, 0])
    assert cache.fork(d, i32([0, 1]), i32([2, 3])).tolist() == [1, 1]
    oracle.fork(MutableLens([16, 13, 0, 0]), [0, 1], [2, 3])
    same(cache, oracle)
    assert sv.sv_query_status(cache.ws) == (sv.SV_OK, 0)


def test_many_pairs_with_and_without_holes():
    n, rows = 300, 600
    lens = [(i * 7) % 41 for i in range(n)]
    cache, oracle = filled(lens, rows, 6, pages=2000)
    bad = [i for i in range(n) if i % 3 == 0 and lens[i] > 0]
    for i in bad:
        hole(cache, oracle, i, (i // 3) % -(-lens[i] // PS))
    d = i32(lens + [0] * n)
    ok = cache.fork(d, i32(range(n)), i32(range(n, rows)))
    good = [i for i in range(n) if i not in bad]
    full = MutableLens(lens + [0] * n)
    oracle.fork(full, good, [n + i for i in good])
    assert ok.tolist() == [int(i not in bad) for i in range(n)] and d.tolist() == list(full)
    assert sv.sv_query_status(cache.ws)[1] == sv.SV_DEV_BAD_PAGE
    same(cache, oracle)
    assert torch.equal(cache.page_refs.cpu(), torch.tensor(oracle.refs))
