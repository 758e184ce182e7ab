"""The oracles of sampling, the paged cache and tree attention on examples worked out by hand, and against
independent dense formulations."""
import numpy as np
import pytest

from oracle.attention import path_of, tree_attention
from oracle.cache import Cache
from oracle.sample import sample_row

LN2 = np.log(2.0)


# ---- sampling: five tokens of weights 1, 1/2, 1/4, 1/4, 0 ------------------------------------------------
X = np.array([-1.0, 0.0, -2.0, -2.0, -np.inf]) * LN2   # order: 1, 0, 2, 3


@pytest.mark.parametrize("T,k,p,q,kept", [
    (1, 0, 1.0, 0.0, [0, 1, 2, 3]),
    (1, 3, 1.0, 0.0, [0, 1, 2]),          # of the equal logits the lower index
    (1, 1, 1.0, 0.0, [1]),
    (1, 9, 1.0, 0.0, [0, 1, 2, 3]),       # a masked token is never kept
    (1, 0, 0.5, 0.0, [1]),                # mass before token 0 is 1/2: not below p
    (1, 0, 0.51, 0.0, [0, 1]),
    (1, 0, 0.8, 0.0, [0, 1, 2]),
    (1, 2, 0.7, 0.0, [0, 1]),             # of the top two: 2/3 before token 0
    (1, 2, 0.66, 0.0, [1]),
    (1, 0, 1.0, 0.3, [0, 1]),
    (2, 0, 1.0, 0.6, [0, 1]),             # weights 2^(-1/2) and 1/2
    (0, 0, 0.1, 0.9, [1]),
])
def test_kept_tokens(T, k, p, q, kept):
    r = sample_row(X, T, k, p, q, [0.0])
    assert list(np.nonzero(r["kept"])[0]) == kept


def test_draws_in_vocabulary_order():
    r = sample_row(X, 1, 0, 1.0, 0.0, [0.0, 0.2, 0.26, 0.7, 0.76, 0.9])   # edges at 1/4, 3/4, 7/8
    assert list(r["tokens"]) == [0, 0, 1, 1, 2, 3]
    assert np.allclose(r["probs"], [0.25, 0.25, 0.5, 0.5, 0.125, 0.125])
    r = sample_row(X, 1, 2, 1.0, 0.0, [0.3, 0.34])                       # edge at 1/3
    assert list(r["tokens"]) == [0, 1] and np.allclose(r["probs"], [1 / 3, 2 / 3])
    r = sample_row(X, 0, 0, 1.0, 0.0, [0.0, 0.999])
    assert list(r["tokens"]) == [1, 1] and list(r["probs"]) == [1, 1]
    r = sample_row(np.full(3, -np.inf), 1, 0, 1.0, 0.0, [0.5])
    assert list(r["tokens"]) == [-1] and list(r["probs"]) == [0]


def test_near_edges_are_told():
    assert list(sample_row(X, 1, 0, 1.0, 0.0, [0.25, 0.3])["near_draw"]) == [True, False]
    assert 0 in sample_row(X, 1, 0, 0.5, 0.0, [0.0])["near_cut"]
    assert len(sample_row(X, 1, 0, 0.6, 0.0, [0.0])["near_cut"]) == 0


# ---- attention ------------------------------------------------------------------------------------------
def test_paths():
    assert path_of(None, 3) == [0, 1, 2, 3]
    assert path_of([-1, 0, 0, 2], 3) == [0, 2, 3]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 0), (3, 2), (4, 9), (99, 1)])
def test_attention_against_a_dense_mask(window, sinks):
    rng = np.random.default_rng(window * 10 + sinks)
    ps, Hq, Hk, D = 4, 4, 2, 3
    lens, offsets, parent = [5, 0], [0, 4, 6], np.array([-1, 0, 0, 2, -1, 0])
    table = np.array([[3, 0, 5], [1, -1, -1]])
    k, v = rng.standard_normal((2, 6, ps, Hk, D))
    q = rng.standard_normal((6, Hq, D))
    out, lse = tree_attention(q, k, v, table, lens, offsets, parent, 0.7, window, sinks)
    # by hand: (position, visible) of each slot per node
    seen = {0: [0], 1: [0, 1], 2: [0, 2], 3: [0, 2, 3]}
    for i, L in enumerate(lens):
        for c in range(offsets[i + 1] - offsets[i]):
            row, here = offsets[i] + c, L + len(seen[c]) - 1
            position = {s: s for s in range(L)} | {L + n: L + d for d, n in enumerate(seen[c])}
            slots = [s for s, p in position.items() if window == 0 or p > here - window or p < sinks]
            for h in range(Hq):
                kk = np.stack([k[table[i, s // ps], s % ps, h // 2] for s in slots])
                vv = np.stack([v[table[i, s // ps], s % ps, h // 2] for s in slots])
                w = np.exp(0.7 * kk @ q[row, h])
                assert np.allclose(out[row, h], w @ vv / w.sum(), rtol=1e-12, atol=1e-13)
                assert np.isclose(lse[row, h], np.log(w.sum()), rtol=1e-12)


# ---- cache ----------------------------------------------------------------------------------------------
def make(pages=6, rows=3, width=3, ps=2, layers=2):
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, layers, pages, ps, 1, 2))
    return Cache(k, v, np.zeros(pages, int), np.full((rows, width), -1))


def test_a_turn_by_hand():
    c = make()
    assert list(c.reserve([0, 0], [3, 2])) == [1, 1]
    assert c.table.tolist() == [[0, 1, -1], [2, -1, -1], [-1, -1, -1]]
    assert c.refs.tolist() == [1, 1, 1, 0, 0, 0]
    new = np.arange(2 * 5 * 2.0).reshape(2, 5, 1, 2)
    c.append(new, -new, [0, 0], [0, 3, 5])
    assert (c.k[:, 0, 0] == new[:, 0]).all() and (c.k[:, 1, 0] == new[:, 2]).all() and (c.v[:, 2, 1] == -new[:, 4]).all()
    # request 0 keeps its root and node 2 (moved to slot 1), request 1 its root
    assert list(c.commit([0, 0], np.array([[2, -1], [-1, -1]]), [1, 0])) == [2, 1]
    assert (c.k[:, 0, 1] == new[:, 2]).all()
    assert c.table.tolist() == [[0, -1, -1], [2, -1, -1], [-1, -1, -1]]
    assert c.refs.tolist() == [1, 0, 1, 0, 0, 0]


def test_refusals_take_nothing():
    c = make(pages=3)
    assert list(c.reserve([0, 0, 0], [4, 4, 2])) == [1, 0, 0]   # two of three pages; then two asked for, one there
    assert c.refs.tolist() == [1, 1, 0]
    assert list(c.reserve([4, 0], [0, 99])) == [1, 0]           # nothing lacks; too wide
    assert c.refs.tolist() == [1, 1, 0]


def test_forks_share_full_pages():
    c = make()
    lens = np.array([0, 0, 0])
    c.reserve([0], [3])
    lens[0] = 3
    assert list(c.fork(lens, [0, 0], [1, 2])) == [1, 1]
    assert c.table.tolist() == [[0, 1, -1], [0, 2, -1], [0, 3, -1]]
    assert c.refs.tolist() == [3, 1, 1, 1, 0, 0] and lens.tolist() == [3, 3, 3]
    assert (c.k[:, 2, 0] == c.k[:, 1, 0]).all() and (c.v[:, 3, 0] == c.v[:, 1, 0]).all()
    c.release(lens, [0, 2])
    assert c.refs.tolist() == [1, 0, 1, 0, 0, 0] and lens.tolist() == [0, 3, 0]
    assert c.table.tolist() == [[-1] * 3, [0, 2, -1], [-1] * 3]
