"""sv_tree_attention where two heads of 64 dimensions make a tile, where they do not, and where row tiles are many and
short, against the float64 oracle (bounds as in test_gpu_attention.py)."""
import os
import sys

import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_attention import _gpu, case, check  # noqa: E402, F401

pytestmark = pytest.mark.gpu


# rows per head of the 16-node trees: 16 (four copies), 32 (two), 64 (one); of the 17-node chain 68: not paired
@pytest.mark.parametrize("Hq,Hk", [(2, 2), (8, 4), (16, 4), (8, 2), (6, 6), (3, 3)])
@pytest.mark.parametrize("tree", ["one", "mixed", "chain"])
@pytest.mark.parametrize("layout", ["slots", "heads"])
def test_heads_of_64(Hq, Hk, tree, layout):
    lens = [0, 1, 17, 113, 127, 128, 300]
    c = case(lens, [tree] * len(lens), Hq, Hk, 64, 16, layout=layout, seed=Hq + Hk)
    check(c)
    check(c, window=40, sinks=3)


@pytest.mark.parametrize("Hq,Hk", [(2, 2), (4, 2), (8, 2)])
def test_a_paired_row_tile_is_split_and_joined(Hq, Hk):
    c = case([5000], ["mixed"], Hq, Hk, 64, 64, seed=Hq)
    check(c)
    c = case([2000, 0, 3001], ["mixed", "one", "wide"], Hq, Hk, 64, 32, seed=Hq)
    check(c, window=1500, sinks=4)


def test_the_heads_of_a_pair_do_not_mix():
    # one head's keys and values far larger than its neighbour's
    c = case([200, 90], ["mixed", "one"], 4, 4, 64, 16, seed=5)
    out = sv.tree_attention(c["q"], c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"])[0].clone()
    c["cache"].k[..., 1, :].mul_(100.0)
    c["cache"].v[..., 1, :].mul_(1e30)
    again = sv.tree_attention(c["q"], c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"])[0]
    assert torch.equal(out[:, [0, 2, 3]], again[:, [0, 2, 3]])


@pytest.mark.parametrize("D,Hq,Hk", [(128, 8, 4), (64, 4, 4)])
@pytest.mark.parametrize("B", [1, 40, 400])
def test_many_short_requests(D, Hq, Hk, B):
    lens = [(i * 37) % 150 for i in range(B)]
    trees = [("one", "none", "mixed", "wide", "chain")[i % 5 if B > 1 else 2] for i in range(B)]
    c = case(lens, trees, Hq, Hk, D, 16, seed=B)
    a, la = check(c)
    b, lb = check(c)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_one_long_request_among_short_ones():
    c = case([6000] + [9] * 60, ["mixed"] + ["one"] * 60, 4, 2, 128, 64, seed=2)
    check(c)
