"""PagedCache.reorder on the GPU against the list-based oracle."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from oracle.cache import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def make(lens, extra, pages, ps=8, layers=2, heads=1, dim=64, width=None, refs_offset=0):
    """Rows of the given lengths, their pages scattered, `extra` slots more reserved."""
    rng = np.random.default_rng(len(lens))
    held = [-(-(n + e) // ps) for n, e in zip(lens, extra)]
    table = np.full((len(lens), width or max(held) + 1), -1)
    order, at = rng.permutation(pages), 0
    for i, n in enumerate(held):
        table[i, :n] = order[at:at + n]
        at += n
    refs = np.zeros(pages, np.int64)
    refs[order[:at]] = 1
    k, v = (torch.randn((layers, pages, ps, heads, dim), device="cuda").to(torch.bfloat16) for _ in range(2))
    d_refs = torch.zeros(pages + refs_offset, dtype=torch.int32, device="cuda")[refs_offset:]
    d_refs.copy_(i32(refs))
    cache = sv.PagedCache(k, v, d_refs, i32(table))
    return cache, Cache(bits(k).copy(), bits(v).copy(), refs, table), i32(lens), np.asarray(lens, np.int64)


def same(cache, oracle, d_len, lens):
    assert np.array_equal(d_len.cpu().numpy(), lens)
    assert np.array_equal(cache.page_table.cpu().numpy(), oracle.table)
    assert np.array_equal(cache.page_refs.cpu().numpy(), oracle.refs)
    assert np.array_equal(bits(cache.k), oracle.k) and np.array_equal(bits(cache.v), oracle.v)


LENS = [0, 1, 7, 8, 9, 15, 16, 17, 30, 40]


@pytest.mark.parametrize("src", [
    list(range(10)), list(range(9, -1, -1)), [9] * 10, [0] * 10, [-1] * 10, [4, 4, 2, 3, 4, 5, 7, 7, 2, -1],
    [1, 2, 3, 4, 5, 6, 7, 8, 9, 0], [3, 3, 3, 1, 1, 1, 8, 8, 8, 8], [1, 0, 3, 2, 5, 4, 6, 6, 9, 9]])
@pytest.mark.parametrize("extra", [0, 3, 20])
def test_maps(src, extra):
    cache, oracle, d_len, lens = make(LENS, [extra] * 10, 80)
    for _ in range(3):                              # the same step again: from what the step before left
        ok = cache.reorder(d_len, i32(src))
        assert int(ok) == oracle.reorder(lens, src) == 1
        same(cache, oracle, d_len, lens)
    assert sv.sv_query_status(cache.ws) == (sv.SV_OK, 0)


def test_random_steps_with_growth():
    rng = np.random.default_rng(5)
    cache, oracle, d_len, lens = make([5] * 24, [0] * 24, 200, width=12, refs_offset=1)
    for _ in range(12):
        more = rng.integers(0, 4, 24)
        more[lens + more > 90] = 0
        assert np.array_equal(cache.reserve(d_len, i32(more)).cpu().numpy(), oracle.reserve(lens, more))
        lens += more
        d_len += i32(more)
        src = rng.integers(0, 24, 24)
        ok = cache.reorder(d_len, i32(src))
        assert int(ok) == oracle.reorder(lens, src)
        same(cache, oracle, d_len, lens)


def test_many_rows():
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 30, 1500)
    cache, oracle, d_len, lens = make(list(lens), [0] * 1500, 9000, layers=1, width=37)
    src = rng.integers(-1, 1500, 1500)
    assert int(cache.reorder(d_len, i32(src))) == oracle.reorder(lens, src) == 1
    same(cache, oracle, d_len, lens)


def test_all_or_nothing():
    cache, oracle, d_len, lens = make([12, 9, 8, 3], [0] * 4, 7)              # 2 + 2 + 1 + 1 pages: one is free
    # two copies of row 0 and of row 1: rows 2 and 3 give back two pages, four are wanted of three
    assert int(cache.reorder(d_len, i32([0, 1, 0, 1]))) == oracle.reorder(lens, [0, 1, 0, 1]) == 1
    same(cache, oracle, d_len, lens)
    cache, oracle, d_len, lens = make([12, 9, 10, 3], [0] * 4, 7)             # 2 + 2 + 2 + 1: none
    for src in ([0, 0, 2, 3], [1, 1, 0, 3], [2, 2, 2, 0]):
        cache, oracle, d_len, lens = make([12, 9, 10, 3], [0] * 4, 7)
        want = oracle.reorder(lens, src)
        assert int(cache.reorder(d_len, i32(src))) == want
        same(cache, oracle, d_len, lens)
        assert sv.sv_query_status(cache.ws)[1] == (0 if want else sv.SV_DEV_OUT_OF_PAGES)
    tight, oracle, d_len, lens = make([12, 12, 16, 16], [0] * 4, 8)           # all held
    src = [0, 0, 0, 2]                                                        # rows 1 and 3 give four back, two are wanted
    assert int(tight.reorder(d_len, i32(src))) == oracle.reorder(lens, src) == 1
    same(tight, oracle, d_len, lens)


@pytest.mark.parametrize("src,status", [([0, 1, 3], "SV_DEV_BAD_SEQ"), ([0, -2, 1], "SV_DEV_BAD_SEQ"), ([2, 2, 1], "SV_DEV_BAD_PAGE"),
                                        ([1, 1, 1], "SV_DEV_BAD_SEQ")])
def test_what_cannot_be_done_changes_nothing(src, status):
    cache, oracle, d_len, lens = make([12, 9, 20], [0] * 3, 12)
    if src == [1, 1, 1]:
        d_len[1] = -3
    cache.page_table[2, 1] = -1                                               # row 2 lacks a page for its slots
    before = [t.clone() for t in (cache.page_table, cache.page_refs, d_len, cache.k, cache.v)]
    assert int(cache.reorder(d_len, i32(src))) == 0
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.page_table, cache.page_refs, d_len, cache.k, cache.v)))
    assert sv.sv_query_status(cache.ws)[1] == getattr(sv, status)
    # rows that nothing names may be in any state
    if src == [2, 2, 1]:
        assert int(cache.reorder(d_len, i32([0, 1, 1]))) == 1


def test_captured_and_replayed():
    cache, oracle, d_len, lens = make([12, 9, 20, 5], [0] * 4, 30)
    src = i32([1, 1, 0, 2])
    ok = i32([0])
    side = torch.cuda.Stream()
    state = [t.clone() for t in (cache.page_table, cache.page_refs, d_len)]
    with torch.cuda.stream(side):
        cache.reorder(d_len, src, ok=ok)
        torch.cuda.synchronize()
        for t, s in zip((cache.page_table, cache.page_refs, d_len), state):
            t.copy_(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cache.reorder(d_len, src, ok=ok)
    torch.cuda.synchronize()
    oracle.k, oracle.v = bits(cache.k).copy(), bits(cache.v).copy()
    for s in ([1, 1, 0, 2], [3, 2, 1, 0], [0, 0, 0, 0]):
        src.copy_(i32(s))
        graph.replay()
        torch.cuda.synchronize()
        assert int(ok) == oracle.reorder(lens, s) == 1
        same(cache, oracle, d_len, lens)


def test_wide_tables():
    """Tables too wide for one CTA, with pages in their first entries only."""
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 60, 30)
    cache, oracle, d_len, lens = make(list(lens), [0] * 30, 400, layers=1, width=2000)
    for _ in range(3):
        src = rng.integers(-1, 30, 30)
        assert int(cache.reorder(d_len, i32(src))) == oracle.reorder(lens, src) == 1
        same(cache, oracle, d_len, lens)
    cache, oracle, d_len, lens = make([30, 30, 40], [0] * 3, 14, width=9000)    # 4 + 4 + 5 pages: one is free
    assert int(cache.reorder(d_len, i32([0, 0, 0]))) == oracle.reorder(lens, [0, 0, 0]) == 1
    same(cache, oracle, d_len, lens)
    cache, oracle, d_len, lens = make([30, 30, 40], [0] * 3, 13, width=9000)    # none
    assert int(cache.reorder(d_len, i32([0, 1, 0]))) == oracle.reorder(lens, [0, 1, 0]) == 1
    cache, oracle, d_len, lens = make([30, 30, 32, 0], [0] * 4, 12, width=9000)
    assert int(cache.reorder(d_len, i32([0, 1, 2, 1]))) == oracle.reorder(lens, [0, 1, 2, 1]) == 0
    same(cache, oracle, d_len, lens)
    assert sv.sv_query_status(cache.ws)[1] == sv.SV_DEV_OUT_OF_PAGES


def test_wider_tables():
    """The same past what one CTA's shared memory holds."""
    cache, oracle, d_len, lens = make([30, 30, 40], [0] * 3, 14, width=20000)   # 4 + 4 + 5 pages: one is free
    assert int(cache.reorder(d_len, i32([0, 0, 0]))) == oracle.reorder(lens, [0, 0, 0]) == 1
    same(cache, oracle, d_len, lens)
    cache, oracle, d_len, lens = make([30, 30, 32, 0], [0] * 4, 12, width=20000)
    assert int(cache.reorder(d_len, i32([0, 1, 2, 1]))) == oracle.reorder(lens, [0, 1, 2, 1]) == 0
    same(cache, oracle, d_len, lens)
    assert sv.sv_query_status(cache.ws)[1] == sv.SV_DEV_OUT_OF_PAGES
