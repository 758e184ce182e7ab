"""The oracles of beam selection, reordering and the 4-bit format on examples worked out by hand."""
import numpy as np

from oracle import quant
from oracle.beam import beam_select
from oracle.cache import Cache

LN2 = np.log(2.0)


def test_two_beams():
    # probabilities 1/2, 1/4, 1/4 and 1/8, 3/8, 1/2: totals of the second beam are half of its own
    x = np.log([[2.0, 1, 1], [1, 3, 4]])
    scores, rows, tokens = beam_select(x, np.array([[0.0, -LN2]]), 6)
    assert np.allclose(np.exp(scores[0]), [1 / 2, 1 / 4, 1 / 4, 1 / 4, 3 / 16, 1 / 16])
    assert list(rows[0]) == [0, 0, 0, 1, 1, 1] and list(tokens[0]) == [0, 1, 2, 2, 1, 0]


def test_finished_missing_and_masked():
    x = np.array([[0.0, 0], [0, -np.inf], [5, 5], [1, 1]])
    scores, rows, tokens = beam_select(x, np.array([[-1.0, -2, -3, -np.inf]]), 5, np.array([[0, 0, 1, 0]]), pad=7)
    assert list(rows[0]) == [0, 0, 1, 2, -1] and list(tokens[0]) == [0, 1, 0, 7, -1]
    assert np.allclose(scores[0][:4], [-1 - LN2, -1 - LN2, -2, -3]) and scores[0][4] == -np.inf


def test_requests_have_rows_of_their_own():
    scores, rows, tokens = beam_select(np.zeros((4, 2)), np.array([[0.0, -9], [-9, 0]]), 2)
    assert rows.tolist() == [[0, 0], [3, 3]] and tokens.tolist() == [[0, 1], [0, 1]]


def cache():
    k = np.arange(6 * 4).reshape(1, 6, 4, 1, 1)
    return Cache(k.copy(), -k, np.array([1, 1, 1, 1, 0, 0]), np.array([[0, 1, -1], [2, 3, -1], [-1, -1, -1]]))


def test_reorder():
    c, lens = cache(), np.array([6, 8, 0])
    assert c.reorder(lens, [0, 0, 1]) == 1          # row 1's pages stay: row 2 goes on from it
    assert c.table.tolist() == [[0, 1, -1], [0, 4, -1], [2, 3, -1]] and list(lens) == [6, 6, 8]
    assert list(c.refs) == [2, 1, 1, 1, 1, 0] and list(c.k[0, 4, :2].flatten()) == [4, 5]
    assert c.reorder(lens, [2, 2, 2]) == 1          # a full last page is shared; pages 0, 1 and 4 are free again
    assert c.table.tolist() == [[2, 3, -1]] * 3 and list(c.refs) == [0, 0, 3, 3, 0, 0]
    assert c.reorder(lens, [-1, 0, -1]) == 1 and list(lens) == [0, 8, 0] and list(c.refs) == [0, 0, 1, 1, 0, 0]


def test_reorder_needs_pages():
    c, lens = cache(), np.array([6, 7, 0])
    c.refs[4:] = 1
    before = c.table.copy()
    assert c.reorder(lens, [0, 1, 0]) == 0 and np.array_equal(c.table, before) and list(lens) == [6, 7, 0]
    assert c.reorder(lens, [0, 0, 0]) == 1          # row 1's pages come free: 2 and 3
    assert c.table.tolist() == [[0, 1, -1], [0, 2, -1], [0, 3, -1]]


def test_codes():
    x = np.array([6, 5, 4.99, 0.25, 0.26, -0.75, 1.25, -1.75, 2.5, 3.5, 0, -0.0, -6, 0.2, 3, -2], np.float32)
    codes, scale = quant.quantise16(x, 1.0)
    assert quant.E4M3[scale] == 1 and list(codes) == [7, 6, 6, 0, 1, 10, 2, 12, 4, 6, 0, 8, 15, 0, 5, 12]
    codes, scale = quant.quantise16(np.zeros(16), 1.0)
    assert scale == 0 and not codes.any()
    assert quant.E4M3[quant.quantise16(np.full(16, 1e9), 1.0)[1]] == 448
    assert quant.E4M3[quant.quantise16(np.full(16, 6 * 2.0 ** -9), 1.0)[1]] == 2.0 ** -9   # the smallest scale


def test_pages_hold_what_was_written():
    g = np.random.default_rng(0)
    for D in (64, 128):
        page, x = np.zeros((1, 1, 16 * 9 * D // 8), np.int64), g.normal(size=(16, D)).astype(np.float32)
        for slot in range(16):
            quant.write(page[0, 0], D, slot, x[slot], False, 0.5)
            quant.write(page[0, 0], D, slot, -x[slot], True, 0.5)
        k, v = quant.read(page, D, 16, 0.5, False)[0, :, 0], quant.read(page, D, 16, 0.5, True)[0, :, 0]
        assert np.array_equal(k, -v)
        # a code is off by at most 1 of its scale (between 4 and 6), the scale by 2^-4 of itself
        top = np.abs(x.reshape(16, -1, 16)).max(-1).repeat(16, 1).reshape(16, D)
        assert (np.abs(k - x) <= top / 6 * (1 + 2.0 ** -4) * 1.5).all()
