"""Tree attention of good requests leaves its status word empty: the sweeps over lengths, windows and batches again, with the
workspace that the call used."""
import os
import sys

import pytest

import speculative_decoding_verification_74_gb300 as sv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_attention import EDGES, _gpu, case, check  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def quiet(c, **kw):
    ws = sv.attention_workspace(c["cache"], c["q"].shape[1])
    check(c, ws=ws, **kw)
    assert sv.sv_query_status(ws) == (sv.SV_OK, 0)


@pytest.mark.parametrize("Hq,Hk,D,ps", [(8, 2, 128, 16), (4, 4, 64, 8), (10, 2, 64, 32), (16, 1, 128, 64), (3, 3, 128, 128),
                                        (8, 1, 64, 256)])
@pytest.mark.parametrize("tree", ["one", "mixed", "chain"])
def test_lengths_at_every_edge(Hq, Hk, D, ps, tree):
    c = case(EDGES, [tree] * len(EDGES), Hq, Hk, D, ps, seed=Hq)
    quiet(c)
    if tree == "chain":
        quiet(c, parent=None)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 4), (100, 200), (129, 1), (10 ** 6, 0)])
def test_windows(window, sinks):
    lens = [0, 1, 4, 127, 128, 129, 260, 513, 700]
    quiet(case(lens, ["mixed"] * len(lens), 4, 2, 64, 16, seed=window), window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128])
def test_mixed_batches(D):
    c = case([40, 0, 500, 3, 700, 129, 1, 0], ["one", "big", "none", "deep", "mixed", "wide", "chain", "none"], 12, 3, D, 16, seed=4)
    quiet(c)
    quiet(c, window=20, sinks=3)


def test_a_long_context():
    quiet(case([6000] + [9] * 20, ["mixed"] + ["one"] * 20, 4, 2, 128, 64, seed=2))
