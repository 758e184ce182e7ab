"""sv_beam_select on the GPU against the float64 oracle: rows and tokens exactly, scores to half a step of float32 (2^-24
of the value) and what the sums of float32 terms leave, 2^-18."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from oracle.beam import beam_select

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def check(logits, scores, K, finished=None, pad=0, ws=None):
    logits, scores = logits.cuda(), scores.cuda()
    fin = None if finished is None else finished.int().cuda()
    got, rows, tokens = sv.beam_select(logits, scores, K, finished=fin, pad=pad, ws=ws)
    want = beam_select(logits.double().cpu().numpy(), scores.double().cpu().numpy(), K,
                       None if finished is None else finished.numpy(), pad)
    assert np.array_equal(rows.cpu().numpy(), want[1])
    assert np.array_equal(tokens.cpu().numpy(), want[2])
    got = got.double().cpu().numpy()
    fine = np.isfinite(want[0])
    assert np.array_equal(np.isfinite(got), fine) and (got[~fine] == -np.inf).all()
    assert (np.abs(got[fine] - want[0][fine]) <= 2.0 ** -24 * np.abs(want[0][fine]) + 2.0 ** -18).all()


def made(B, W, V, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B * W, V), generator=g) * spread).to(dtype), -10 - 3 * torch.rand((B, W), generator=g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,W,V,K", [(1, 1, 1, 1), (3, 1, 2, 5), (2, 4, 3, 128), (1, 4, 32000, 8), (3, 3, 1001, 6), (2, 5, 4099, 33),
                                     (5, 2, 20000, 1), (1, 64, 500, 128), (1, 33, 777, 64), (40, 8, 300, 16), (1, 2, 151937, 100)])
def test_sizes(dtype, B, W, V, K):
    check(*made(B, W, V, dtype, V + K), K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lead", range(9))
def test_strides_and_alignment(dtype, lead):
    x, scores = made(2, 3, 9001, dtype, lead)
    wide = torch.full((6, 9001 + 13), 50.0, dtype=dtype, device="cuda")
    wide[:, lead:lead + 9001] = x.cuda()
    logits = wide[:, lead:lead + 9001]
    # the float32 sums group the logits by where they lie: scores agree as far as each agrees with the oracle
    check(logits, scores, 9)
    check(x, scores, 9)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [1, 8, 100, 128])
def test_runs_of_equals(dtype, K):
    """Constant rows, rising and falling ones, long runs of the largest logit: ties go to the lowest token."""
    V = 40000
    x = torch.zeros((8, V))
    x[1] = torch.arange(V) / 1000.0
    x[2] = -torch.arange(V) / 1000.0
    x[3, 20000:] = 1
    x[4, ::2] = 1
    x[5, -5:] = 3
    x[6] = (torch.arange(V) % 7).float()
    x[7, 100:140] = -1
    for i in range(8):
        check(x[i:i + 1].to(dtype), torch.tensor([[-1.5]]), K)
    check(x.to(dtype), torch.linspace(-3, -1, 8)[None, :].contiguous(), K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scores_in_place(dtype):
    """The new scores over the old ones, also where equal totals of two beams have their rows summed again."""
    x, scores = made(3, 4, 5000, dtype, 5)
    x[1], x[6] = x[0], x[5]
    scores[0, 1], scores[1, 2] = scores[0, 0], scores[1, 1]
    want = sv.beam_select(x.cuda(), scores.cuda(), 4)
    place, ints = scores.cuda(), torch.empty((2, 3, 4), dtype=torch.int32, device="cuda")
    got = sv.beam_select(x.cuda(), place, 4, out=(place, ints[0], ints[1]))
    assert got[0] is place
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_equal_beams():
    """Beams with the same logits and scores: every total occurs twice or more, the lower beam first."""
    x, scores = made(2, 4, 5000, torch.float32, 1)
    x[1], x[2], x[6] = x[0], x[0], x[5]
    scores[0, :3], scores[1, 1:3] = -4.0, -5.0
    check(x, scores, 30)
    check(x.to(torch.bfloat16), scores, 30)


def test_totals_that_lie_close_together():
    """Beams whose best totals differ by 2^-21 to 2^-27, less than float32 sums can tell."""
    g = torch.Generator().manual_seed(3)
    base = torch.randn(3000, generator=g, dtype=torch.float64)
    for step in (2.0 ** -21, 2.0 ** -24, 2.0 ** -27):
        x = torch.stack([base.float()] * 6)
        x[:, 100] = 9.0                              # the same best token; the rest moves the sum by a little
        for w in range(6):
            x[w, 200] = float(np.log(1000 + [3, 5, 0, 4, 1, 2][w] * step * 40000))
        check(x, torch.full((1, 6), -2.0), 6)


def test_masked_logits_and_missing_beams():
    x, scores = made(3, 4, 6000, torch.float32, 2)
    x[0] = -torch.inf                                # a beam without a token
    x[1, :5990] = -torch.inf                         # ten tokens left
    x[2, 5:] = -torch.inf
    x[4:8] = -torch.inf
    x[5, 4321] = 2.0                                 # one candidate in all
    x[9, ::2] = -torch.inf
    x[10] = -3.4e38
    scores[2, 1] = scores[0, 3] = -torch.inf
    check(x, scores, 40)
    x, scores = made(2, 3, 50, torch.bfloat16, 4)
    scores[0] = -torch.inf                           # no beam at all
    check(x, scores, 4)


def test_finished_beams():
    x, scores = made(4, 4, 3000, torch.bfloat16, 6)
    finished = torch.tensor([[0, 1, 0, 0], [1, 1, 1, 1], [0, 0, 0, 1], [1, 0, 1, 0]])
    scores[0, 1], scores[3, 0], scores[3, 2] = -10.5, -torch.inf, scores[3, 1]
    x[1] = float("nan")                              # not looked at
    x[4:8] = float("inf")
    clean = x.clone()
    clean[1], clean[4:8] = 0, 0
    for pad in (0, 2999, 2 ** 30):
        check(clean, scores, 8, finished, pad)
        a = sv.beam_select(x.cuda(), scores.cuda(), 8, finished=finished.int().cuda(), pad=pad)
        b = sv.beam_select(clean.cuda(), scores.cuda(), 8, finished=finished.int().cuda(), pad=pad)
        assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_logits(dtype):
    x, scores = made(2, 3, 9000, dtype, 8)
    x[0] *= 1e4
    x[1] *= 1e30
    x[2] = 3e38
    x[3, 7] = 200.0
    x[4, 8500] = 1000.0
    check(x, scores, 12)


def test_bad_input_marks_its_request_alone():
    x, scores = made(5, 2, 2000, torch.float32, 9)
    want = sv.beam_select(x.cuda(), scores.cuda(), 4)
    x[2, 1999] = float("nan")
    x[5, 0] = float("inf")
    scores[3, 1] = float("nan")
    ws = sv.beam_workspace(10, 2000, 4)
    got = sv.beam_select(x.cuda(), scores.cuda(), 4, ws=ws)
    assert sv.sv_query_status(ws) == (sv.SV_ERR_DEVICE_INPUT, sv.SV_DEV_BAD_LOGIT)
    for i in (1, 2, 3):
        assert torch.isnan(got[0][i]).all() and (got[1][i] == -1).all() and (got[2][i] == -1).all()
    for i in (0, 4):
        assert all(torch.equal(a[i], b[i]) for a, b in zip(got, want))
    assert sv.sv_query_status(ws) == (sv.SV_OK, 0)


def test_other_stream_and_replay():
    x, scores = made(4, 4, 30000, torch.bfloat16, 10)
    x, scores = x.cuda(), scores.cuda()
    want = sv.beam_select(x, scores, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.beam_select(x, scores, 8, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws, out = sv.beam_workspace(16, 30000, 8), [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.beam_select(x, scores, 8, out=out, ws=ws)
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_equals_over_many_parts_and_beams(dtype):
    """Rows long enough for many parts: constant ones, equal beams, and a step between parts."""
    V = 150000
    x = torch.zeros((8, V))
    x[2:4] = torch.arange(V)[None, :] // 30000.0
    x[4:6, 70000:] = 1.0
    x[6:8] = torch.randn((1, V), generator=torch.Generator().manual_seed(1))
    x = x.to(dtype)
    for K in (1, 33, 128):
        check(x, torch.full((1, 8), -3.0), K)
        check(x, torch.tensor([[-3.0, -3.5], [-3.0, -2.0], [-1.0, -1.0], [-4.0, -4.25]]), K)
