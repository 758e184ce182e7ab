"""The paged cache held in 4 bits on the GPU: its rounding against the format's definition, code by code, and its
bookkeeping against the list-based oracle, whose elements are (code, scale) pairs."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from oracle import quant
from oracle.cache import Cache
from synth.trees import TREE_SHAPES, tree_shape

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def pairs(pool, D, ps, value):
    """[layers, pages, page_size, heads, D] of code + 16 * scale byte."""
    pool = pool.cpu().numpy().astype(np.int64)
    out = np.zeros(pool.shape[:2] + (ps, pool.shape[2], D), np.int64)
    for slot in range(ps):
        at = np.array([quant.places(D, slot, d, value) for d in range(D)])
        code = (pool[..., at[:, 0]] >> (4 * at[:, 1])) & 15
        out[:, :, slot] = code + 16 * pool[..., at[:, 2]]
    return out


def quantised(x, whole_scale):
    """code + 16 * scale byte of every element of a tensor [..., D]."""
    x = x.float().cpu().numpy()
    out = np.zeros(x.shape, np.int64)
    for at in np.ndindex(x.shape[:-1]):
        for d in range(0, x.shape[-1], 16):
            codes, scale = quant.quantise16(x[at][d:d + 16], whole_scale)
            out[at][d:d + 16] = codes + 16 * scale
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("k_scale,v_scale", [(1.0, 1.0), (0.37, 2.0 ** -6), (3.0, 100.0)])
def test_rounding(D, k_scale, v_scale):
    g = torch.Generator().manual_seed(D)
    x = torch.randn((40, 2, D), generator=g)
    x[1] = 0
    x[2] = -0.0
    x[3] *= 1e-3                                   # scales among e4m3's subnormal numbers
    x[4] *= 1e-5                                   # scales of 0
    x[5] *= 3e4                                    # above e4m3's range: saturated
    x[6] = 6 * k_scale                             # ties: with scale 1 halves of a step
    x[6, :, 1:16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.5]) * k_scale
    x[7, :, ::16] = 1e4
    x[8:] *= torch.exp2(torch.randint(-8, 8, (32, 2, D), generator=g).float())
    x = x.to(torch.bfloat16).cuda()
    y = x.flip(0).contiguous()
    cache = sv.PagedCache4.empty(1, 6, 16, 2, D, 2, 4, k_scale=k_scale, v_scale=v_scale)
    lens, offs = i32([5, 3]), i32([0, 20, 40])
    cache.reserve(lens, i32([20, 20]))
    cache.append(x, y, lens, offs)
    assert sv.sv_query_status(cache.ws) == (sv.SV_OK, 0)
    k, v = (pairs(cache.pool, D, 16, value)[0] for value in (False, True))
    table = cache.page_table.cpu().numpy()
    want_k, want_v = quantised(x, k_scale), quantised(y, v_scale)
    for i, n in enumerate([5, 3]):
        for c in range(20):
            page, slot = table[i, (n + c) // 16], (n + c) % 16
            assert np.array_equal(k[page, slot], want_k[20 * i + c])
            assert np.array_equal(v[page, slot], want_v[20 * i + c])
    # what the oracle reads back is the nearest code's value: off by at most half the widest step of its scale
    back = quant.read(cache.pool[0].cpu().numpy(), D, 16, k_scale, False)
    page, slot = table[0, 0], 5
    t = x[0].double().cpu().numpy()
    step = quant.E4M3[k[page, slot] >> 4] * k_scale
    assert (np.abs(back[page, slot] - t) <= 1.0 * step + 2.0 ** -4 * np.abs(t).max()).all()


def test_values_that_are_not_finite_are_reported():
    for bad in (float("nan"), float("inf"), float("-inf")):
        cache = sv.PagedCache4.empty(1, 2, 8, 1, 64, 1, 2)
        x = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
        y = x.clone()
        y[1, 0, 37] = bad
        lens = i32([0])
        cache.reserve(lens, i32([3]))
        cache.append(x, y, lens, i32([0, 3]))
        assert sv.sv_query_status(cache.ws) == (sv.SV_ERR_DEVICE_INPUT, sv.SV_DEV_BAD_VALUE)
        values = quant.read(cache.pool[0].cpu().numpy(), 64, 8, 1.0, True)[int(cache.page_table[0, 0])]
        assert np.isfinite(values).all() and np.allclose(values[[0, 2]], 1, atol=0.07)


def make(layers, pages, ps, heads, dim, rows, width, stride=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = ps * 9 * dim // 8
    pool = torch.randint(0, 256, (layers, pages, heads, n + stride), dtype=torch.uint8, generator=g, device="cuda")[..., :n]
    cache = sv.PagedCache4(pool, torch.zeros(pages, dtype=torch.int32, device="cuda"),
                           torch.full((rows, width), -1, dtype=torch.int32, device="cuda"), ps, dim, k_scale=0.5, v_scale=0.25)
    oracle = Cache(pairs(pool, dim, ps, False), pairs(pool, dim, ps, True), np.zeros(pages, np.int32), np.full((rows, width), -1))
    return cache, oracle


def same(cache, oracle, lens):
    """Tables, counts, and every slot of a sequence."""
    assert np.array_equal(cache.page_table.cpu().numpy(), oracle.table)
    assert np.array_equal(cache.page_refs.cpu().numpy(), oracle.refs)
    ps, D = oracle.ps, cache.head_dim
    for value, want in ((False, oracle.k), (True, oracle.v)):
        got = pairs(cache.pool, D, ps, value)
        for i, n in enumerate(lens):
            slots = np.arange(n)
            pages = oracle.table[i, slots // ps]
            assert np.array_equal(got[:, pages, slots % ps], want[:, pages, slots % ps])


@pytest.mark.parametrize("layers,pages,ps,heads,dim,rows,stride", [
    (1, 40, 8, 1, 64, 5, 0), (3, 64, 16, 2, 128, 7, 16), (2, 200, 8, 3, 64, 20, 32), (2, 41, 64, 2, 128, 4, 0)])
def test_random_rounds(layers, pages, ps, heads, dim, rows, stride):
    rng = np.random.default_rng(layers * 100 + ps)
    width = max(3, 96 // ps)
    cache, oracle = make(layers, pages, ps, heads, dim, rows, width, stride)
    lens = np.zeros(rows, np.int64)
    for rnd in range(5):
        shapes = [tree_shape(*TREE_SHAPES[int(rng.integers(8))]) if rng.random() < 0.85 else np.zeros(0, np.int32)
                  for _ in range(rows)]
        counts = np.asarray([len(s) for s in shapes])
        d_len = i32(lens)
        ok = cache.reserve(d_len, i32(counts))
        want = oracle.reserve(lens, counts)
        assert np.array_equal(ok.cpu().numpy(), want)
        counts = counts * want                      # unserved requests sit the round out
        offs = np.concatenate([[0], np.cumsum(counts)])
        room = [torch.randn((layers, int(offs[-1]) + 1, heads * dim + 8), device="cuda").to(torch.bfloat16) for _ in range(2)]
        new = [r[:, 1:, 8:].unflatten(2, (heads, dim)) for r in room]   # strided rows
        cache.append(new[0], new[1], d_len, i32(offs))
        oracle.append(quantised(new[0], 0.5), quantised(new[1], 0.25), lens, offs)
        same(cache, oracle, lens + counts)
        paths, acc = [], []
        for s, n in zip(shapes, counts):
            node, path = int(rng.integers(len(s))) if n else 0, []
            while node > 0:
                path.append(node)
                node = int(s[node])
            paths.append(path[::-1])
            acc.append(len(path) if n and rng.random() < 0.9 else -1)
        path = np.full((rows, 16), -1)
        for i, p in enumerate(paths):
            path[i, :len(p)] = p
        cache.commit(d_len, i32(offs), i32(path), i32(acc), out_len=d_len)       # lengths in place
        lens = oracle.commit(lens, path, np.asarray(acc))
        assert np.array_equal(d_len.cpu().numpy(), lens)
        same(cache, oracle, lens)
        gone = rng.choice(rows, rows // 3 + 1, replace=False)
        cache.release(d_len, i32(gone))
        oracle.release(lens, gone)
        src = rng.choice(np.setdiff1d(np.arange(rows), gone), len(gone))
        done = cache.fork(d_len, i32(src), i32(gone))
        assert np.array_equal(done.cpu().numpy(), oracle.fork(lens, src, gone))
        same(cache, oracle, lens)
        src = rng.integers(-1, rows, rows)
        ok = cache.reorder(d_len, i32(src))
        assert int(ok) == oracle.reorder(lens, src)
        assert np.array_equal(d_len.cpu().numpy(), lens)
        same(cache, oracle, lens)
    assert sv.sv_query_status(cache.ws)[1] & ~sv.SV_DEV_OUT_OF_PAGES == 0


def test_copies_leave_other_pages_alone():
    """A fork and a reorder write the new pages' used groups of eight slots, and nothing else."""
    cache, oracle = make(2, 12, 16, 2, 128, 4, 3, seed=3)
    lens = i32([20, 0, 0, 0])
    cache.reserve(lens, i32([0, 0, 0, 0]))
    before = cache.pool.clone()
    cache.fork(lens, i32([0]), i32([2]))
    cache.reorder(lens, i32([2, 0, 0, -1]))
    table = cache.page_table.cpu().numpy()
    assert lens.tolist() == [20, 20, 20, 0] and len(set(table[:3, 0])) == 1 and len(set(table[:3, 1])) == 3
    used = 9 * 128
    changed = (cache.pool != before).cpu().numpy()
    untouched = [p for p in range(12) if p not in table[:3, 1]]
    assert not changed[:, untouched].any() and not changed[..., used:].any()
    for p in table[:3, 1]:
        assert torch.equal(cache.pool[:, p, :, :used], before[:, table[1, 1], :, :used])
