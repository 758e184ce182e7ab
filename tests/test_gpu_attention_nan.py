"""A query row that is not finite has no softmax: its outputs are NaN, in row tiles of one CTA and in those that several CTAs
work on, and every other row's are what they were."""
import os
import sys

import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_attention import _gpu, case  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def call(c, q, **kw):
    ws = sv.attention_workspace(c["cache"], q.shape[1])
    out = sv.tree_attention(q, c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"], ws=ws, **kw)
    assert sv.sv_query_status(ws) == (sv.SV_OK, 0)
    return out


# rows of one, two and four copies, paired heads and single ones; few slots (one CTA a row tile) and many (several)
@pytest.mark.parametrize("Hq,Hk,D", [(8, 2, 128), (4, 4, 128), (32, 2, 128), (4, 2, 64), (16, 4, 64), (3, 3, 64), (16, 2, 64)])
@pytest.mark.parametrize("lens,trees", [([0, 40, 127, 300], ["mixed", "one", "wide", "chain"]), ([20011], ["mixed"]),
                                        ([7000, 3, 5000], ["chain", "one", "mixed"])])
@pytest.mark.parametrize("window", [0, 100])
def test_one_row_of_nan(Hq, Hk, D, lens, trees, window):
    c = case(lens, trees, Hq, Hk, D, 64, seed=Hq + D)
    q = c["q"]
    want, want_lse = call(c, q, window=window, sinks=2)
    assert bool(want.isfinite().all()) and bool(want_lse.isfinite().all())
    last = q.shape[0] - 1
    for row, head, whole in ((0, 0, True), (last, Hq - 1, False), (last // 2, Hq // 2, False)):
        bad = q.clone()
        if whole:
            bad[row, head] = float("nan")
        else:
            bad[row, head, (7 * head) % D] = float("nan")
        out, lse = call(c, bad, window=window, sinks=2)
        assert bool(out[row, head].isnan().all()) and bool(lse[row, head].isnan())
        out[row, head], lse[row, head] = want[row, head], want_lse[row, head]
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        alone = call(c, bad, window=window, sinks=2, lse=False)[0]
        assert bool(alone[row, head].isnan().all())


@pytest.mark.parametrize("n", [30, 20011])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_of_minus_infinity_only(n, D):
    """exp(-inf - (-inf)): no softmax either, and a log-sum-exp of -inf."""
    c = case([n], ["mixed"], 4, 2, D, 64, seed=3)
    want, want_lse = call(c, c["q"])
    c["cache"].k[..., 0] = 1.0
    bad = torch.zeros_like(c["q"])
    bad[:, :, 1:] = c["q"][:, :, 1:]
    want, want_lse = call(c, bad)
    bad[5, 2, 0] = -float("inf")
    out, lse = call(c, bad)
    assert bool(out[5, 2].isnan().all()) and lse[5, 2].item() == -float("inf")
    out[5, 2], lse[5, 2] = want[5, 2], want_lse[5, 2]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_bad_requests_still_get_zeros():
    c = case([30, 40], ["mixed", "mixed"], 4, 2, 64, 16, seed=9)
    q = c["q"].clone()
    q[3], q[20] = float("nan"), float("nan")
    c["cache"].page_table[1, 0] = -1
    ws = sv.attention_workspace(c["cache"], 4)
    out, lse = sv.tree_attention(q, c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"], ws=ws)
    assert sv.sv_query_status(ws)[1] == sv.SV_DEV_BAD_PAGE
    assert bool((out[16:] == 0).all()) and bool((lse[16:] == -float("inf")).all())
    assert bool(out[3].isnan().all()) and bool(out[:3].isfinite().all()) and bool(out[4:16].isfinite().all())
