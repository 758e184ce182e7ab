"""The paged cache on the GPU against the list-based oracle: tables, counts, lengths and every bit of the
pools, through random rounds of reserve, append, commit, fork and release."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from oracle.cache import Cache
from synth.trees import TREE_SHAPES, tree_shape

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def make(layers, pages, ps, heads, dim, rows, width, layout="slots", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (layers, pages, ps, heads, dim) if layout == "slots" else (layers, pages, heads, ps, dim)
    k, v = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    if layout == "heads":
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    cache = sv.PagedCache(k, v, refs, table)
    oracle = Cache(bits(k).copy(), bits(v).copy(), refs.cpu().numpy().copy(), table.cpu().numpy().copy())
    return cache, oracle


def same(cache, oracle):
    assert np.array_equal(cache.page_table.cpu().numpy(), oracle.table)
    assert np.array_equal(cache.page_refs.cpu().numpy(), oracle.refs)
    assert np.array_equal(bits(cache.k), oracle.k) and np.array_equal(bits(cache.v), oracle.v)


def random_path(rng, parent):
    node, path = int(rng.integers(len(parent))), []
    while node > 0:
        path.append(node)
        node = int(parent[node])
    return path[::-1]


@pytest.mark.parametrize("layers,pages,ps,heads,dim,rows,layout", [
    (1, 40, 8, 1, 64, 5, "slots"), (3, 64, 16, 2, 128, 7, "heads"), (2, 300, 8, 3, 64, 33, "slots"),
    (5, 41, 64, 8, 128, 4, "slots"), (1, 5000, 8, 1, 64, 40, "heads")])
def test_random_rounds(layers, pages, ps, heads, dim, rows, layout):
    rng = np.random.default_rng(layers * 100 + ps)
    width = max(3, 96 // ps)
    cache, oracle = make(layers, pages, ps, heads, dim, rows, width, layout)
    lens = np.zeros(rows, np.int64)
    for rnd in range(6):
        shapes = [tree_shape(*TREE_SHAPES[int(rng.integers(8))]) if rng.random() < 0.85 else np.zeros(0, np.int32)
                  for _ in range(rows)]
        counts = np.asarray([len(s) for s in shapes])
        d_len = i32(lens)
        ok = cache.reserve(d_len, i32(counts))
        want = oracle.reserve(lens, counts)
        assert np.array_equal(ok.cpu().numpy(), want)
        counts = counts * want                      # unserved requests sit the round out
        shapes = [s if want[i] else s[:0] for i, s in enumerate(shapes)]
        offs = np.concatenate([[0], np.cumsum(counts)])
        new = [torch.randn((layers, int(offs[-1]), heads, dim), device="cuda").to(torch.bfloat16) for _ in range(2)]
        cache.append(new[0], new[1], d_len, i32(offs))
        oracle.append(bits(new[0]), bits(new[1]), lens, offs)
        same(cache, oracle)
        paths = [random_path(rng, s) if len(s) else [] for s in shapes]
        acc = np.asarray([len(p) if len(s) and rng.random() < 0.9 else -1 for p, s in zip(paths, shapes)])
        nmax = max(16, max(len(p) for p in paths))
        path = np.full((rows, nmax), -1)
        for i, p in enumerate(paths):
            path[i, :len(p)] = p
        cache.commit(d_len, i32(offs), i32(path), i32(acc), out_len=d_len)       # lengths in place
        lens = oracle.commit(lens, path, acc)
        assert np.array_equal(d_len.cpu().numpy(), lens)
        same(cache, oracle)
        # some rows end, and their places are taken by copies of others
        gone = rng.choice(rows, rows // 3 + 1, replace=False)
        cache.release(d_len, i32(gone))
        oracle.release(lens, gone)
        same(cache, oracle)
        src = rng.choice(np.setdiff1d(np.arange(rows), gone), len(gone))
        done = cache.fork(d_len, i32(src), i32(gone))
        assert np.array_equal(done.cpu().numpy(), oracle.fork(lens, src, gone))
        assert np.array_equal(d_len.cpu().numpy(), lens)
        same(cache, oracle)
    assert sv.sv_query_status(cache.ws)[1] & ~sv.SV_DEV_OUT_OF_PAGES == 0


def test_pool_exhaustion_serves_rows_in_order():
    cache, oracle = make(1, 10, 8, 1, 64, 6, 8)
    lens, extra = np.zeros(6, int), np.asarray([16, 0, 40, 24, 0, 8])    # 2, 0, 5 pages, then too few
    ok = cache.reserve(i32(lens), i32(extra))
    assert ok.tolist() == oracle.reserve(lens, extra).tolist() == [1, 1, 1, 1, 1, 0]
    same(cache, oracle)
    assert sv.sv_query_status(cache.ws) == (sv.SV_ERR_DEVICE_INPUT, sv.SV_DEV_OUT_OF_PAGES)
    ok = cache.reserve(i32(lens), i32([16, 0, 64, 24, 0, 0]))             # row 2 wants three more: none left
    assert ok.tolist() == oracle.reserve(lens, [16, 0, 64, 24, 0, 0]).tolist() == [1, 1, 0, 1, 1, 1]
    same(cache, oracle)


def test_page_boundaries_and_counts():
    """Lengths at, before and after page edges; a path that skips nodes; a single-token append."""
    for n in (0, 1, 7, 8, 9, 15, 16, 17):
        cache, oracle = make(2, 12, 8, 2, 64, 2, 6, seed=n)
        lens = np.asarray([n, 3])
        assert cache.reserve(i32(lens), i32([5, 1])).tolist() == [1, 1]
        oracle.reserve(lens, [5, 1])
        offs = np.asarray([0, 5, 6])
        new = [torch.randn((2, 6, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2)]
        cache.append(new[0], new[1], i32(lens), i32(offs))
        oracle.append(bits(new[0]), bits(new[1]), lens, offs)
        path = np.asarray([[2, 4, -1, -1, -1], [-1] * 5])
        out = cache.commit(i32(lens), i32(offs), i32(path), i32([2, 0]))
        assert out.tolist() == oracle.commit(lens, path, [2, 0]).tolist() == [n + 3, 4]
        same(cache, oracle)
    # one layer at a time, as a forward pass does
    cache, oracle = make(3, 6, 8, 2, 64, 1, 4)
    cache.reserve(i32([0]), i32([2]))
    oracle.reserve([0], [2])
    for layer in range(3):
        new = [torch.randn((2, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2)]
        cache.append(new[0], new[1], i32([0]), i32([0, 2]), layer=layer)
        oracle.append(bits(new[0])[None], bits(new[1])[None], [0], [0, 2], layer=layer)
    same(cache, oracle)


def test_bad_values_touch_nothing():
    cache, oracle = make(1, 8, 8, 1, 64, 4, 3)
    lens = np.asarray([4, 4, 0, 0])
    cache.reserve(i32([0] * 4), i32([8, 8, 0, 0]))
    oracle.reserve([0] * 4, [8, 8, 0, 0])
    ok = cache.reserve(i32([-1, 4, 0, 0]), i32([1, 100, -2, 0]))
    assert ok.tolist() == [0, 0, 0, 1]
    same(cache, oracle)
    assert sv.sv_query_status(cache.ws) == (sv.SV_ERR_DEVICE_INPUT, sv.SV_DEV_BAD_SEQ)
    # paths: not increasing, past the tree, a length past the tree
    for path, acc in (([2, 2, -1], 2), ([3, -1, -1], 1), ([0, -1, -1], 1), ([1, 2, 2], 3)):
        out = cache.commit(i32(lens), i32([0, 3, 3, 3, 3]), i32([path, [-1] * 3, [-1] * 3, [-1] * 3]), i32([acc, 0, 0, 0]))
        assert out.tolist() == [4, 4, 0, 0]
        assert sv.sv_query_status(cache.ws)[1] == sv.SV_DEV_BAD_SEQ
        same(cache, oracle)
    # forks onto held, missing or doubled rows
    d = i32([8, 8, 0, 0])
    ok = cache.fork(d, i32([0, 0, 0, 0, 9]), i32([1, 7, 2, 2, 3]))
    assert ok.tolist() == [0, 0, 0, 0, 0] and d.tolist() == [8, 8, 0, 0]
    assert sv.sv_query_status(cache.ws)[1] == sv.SV_DEV_BAD_SEQ
    same(cache, oracle)
    # a node whose slot has no page, and rows outside the new keys
    new = torch.ones((1, 30, 1, 64), dtype=torch.bfloat16, device="cuda")
    cache.append(new, new, i32([0, 7, 0, 0]), i32([0, 0, 9, 9, 9]))
    oracle.append(bits(new), bits(new), [0, 7, 0, 0], [0, 0, 1, 1, 1])
    same(cache, oracle)
    assert sv.sv_query_status(cache.ws)[1] == sv.SV_DEV_BAD_PAGE
    cache.append(new, new, i32([0, 0, 0, 0]), i32([0, 0, 0, 0, 31]))
    same(cache, oracle)
    assert sv.sv_query_status(cache.ws)[1] == sv.SV_DEV_BAD_NODES
    # a page given back too often keeps its count at 0
    cache.page_refs.zero_()
    cache.release(d, i32([0, 11]))
    assert torch.all(cache.page_refs == 0) and cache.page_table[0].tolist() == [-1] * 3 and d.tolist() == [0, 8, 0, 0]
    assert sv.sv_query_status(cache.ws)[1] == sv.SV_DEV_BAD_PAGE | sv.SV_DEV_BAD_SEQ
    assert sv.sv_query_status(cache.ws) == (sv.SV_OK, 0)


def test_released_twice_counts_once():
    cache, oracle = make(1, 8, 8, 1, 64, 3, 2)
    cache.reserve(i32([0] * 3), i32([16, 8, 0]))
    d = i32([12, 8, 0])
    cache.fork(d, i32([0]), i32([2]))
    cache.release(d, i32([0, 0, 2]))
    assert cache.page_refs.tolist() == [0, 0, 1, 0, 0, 0, 0, 0] and d.tolist() == [0, 8, 0]
    assert sv.sv_query_status(cache.ws) == (sv.SV_OK, 0)


def test_offsets_past_32_bits():
    """The last pages of a pool of more than 2^32 elements."""
    pages, ps, heads, dim = 32769 + 16, 128, 8, 128            # 131072 elements a page
    k = torch.empty((1, pages, ps, heads, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 32
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[-3:] = 0
    cache = sv.PagedCache(k, v, refs, torch.full((2, 4), -1, dtype=torch.int32, device="cuda"))
    d = i32([0, 0])
    assert cache.reserve(d, i32([140, 0])).tolist() == [1, 1]
    assert cache.page_table[0].tolist() == [pages - 3, pages - 2, -1, -1]
    new = [torch.randn((1, 140, heads, dim), device="cuda").to(torch.bfloat16) for _ in range(2)]
    cache.append(new[0], new[1], d, i32([0, 140, 140]))
    assert torch.equal(k[0, pages - 2, :12], new[0][0, 128:]) and torch.equal(v[0, pages - 3], new[1][0, :128])
    path = torch.full((2, 140), -1, dtype=torch.int32, device="cuda")
    path[0, 0] = 139
    out = cache.commit(d, i32([0, 140, 140]), path, i32([1, 0]), out_len=d)
    assert out.tolist() == [2, 0] and torch.equal(k[0, pages - 3, 1], new[0][0, 139])
    cache.fork(d, i32([0]), i32([1]))
    assert cache.page_table[1].tolist() == [pages - 2, -1, -1, -1] and torch.equal(v[0, pages - 2, 1], new[1][0, 139])


def test_stream_and_graph():
    cache, oracle = make(2, 30, 8, 2, 64, 3, 6)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    lens, extra, offs = i32([0, 5, 9]), i32([4, 4, 4]), i32([0, 4, 8, 12])
    new = [torch.randn((2, 12, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2)]
    path, acc = i32([[1, 3, -1, -1], [2, -1, -1, -1], [-1] * 4]), i32([2, 1, 0])
    ok, out = i32([0] * 3), i32([0] * 3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cache.reserve(lens, extra, ok=ok)
        cache.append(new[0], new[1], lens, offs)
        cache.commit(lens, offs, path, acc, out_len=out)
    for _ in range(2):
        graph.replay()
        oracle.reserve([0, 5, 9], [4, 4, 4])
        oracle.append(bits(new[0]), bits(new[1]), [0, 5, 9], [0, 4, 8, 12])
        assert oracle.commit([0, 5, 9], path.cpu().numpy(), [2, 1, 0]).tolist() == [3, 7, 10]
    torch.cuda.synchronize()
    assert ok.tolist() == [1, 1, 1] and out.tolist() == [3, 7, 10]
    same(cache, oracle)
