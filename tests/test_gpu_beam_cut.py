"""sv_beam_select where equal logits of one beam lie on both sides of the cut, and another beam's total next to them: the order is
that of the exact totals.

The beams of a request hold the same logits in another order, so their log-sums agree exactly; one's score is a step of float32
(2^-26 or more, against 2^-30 of the sums that are told apart) above the others'.  So the better beam's largest logits come
first, in the order of their tokens, then the others', the lower beam before the higher one."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def made(requests, W, V, equals, top, dtype, seed, score):
    g = torch.Generator().manual_seed(seed)
    x, tokens = torch.empty((requests, W, V), dtype=dtype), torch.empty((requests, W, equals), dtype=torch.int64)
    for i in range(requests):
        row = torch.randn(V, generator=g).to(dtype)
        row[:equals] = top
        for w in range(W):
            order = torch.randperm(V, generator=g)
            x[i, w] = row[order]
            tokens[i, w] = torch.nonzero(order < equals)[:, 0]
    better = torch.randint(W, (requests,), generator=g)
    scores = torch.full((requests, W), score)
    scores[torch.arange(requests), better] = float(np.nextafter(np.float32(score), np.float32(np.inf)))
    return x.reshape(requests * W, V), scores, better, tokens


def check(requests, W, V, equals, top, dtype, seed, score, K):
    x, scores, better, tokens = made(requests, W, V, equals, top, dtype, seed, score)
    got, rows, picked = sv.beam_select(x.cuda(), scores.cuda(), K)
    for i in range(requests):
        order = [int(better[i])] + [w for w in range(W) if w != int(better[i])]
        want = [(i * W + w, int(v)) for w in order for v in tokens[i, w]][:K]
        assert list(zip(rows[i].tolist(), picked[i].tolist())) == want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [6.0, 25.0])
@pytest.mark.parametrize("equals,K", [(2, 1), (3, 2), (7, 3), (12, 8)])
def test_equals_of_one_beam_around_the_cut(dtype, top, equals, K):
    check(240, 2, 20001, equals, top, dtype, equals, 0.2, K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W,equals,K", [(2, 200, 64), (3, 170, 128), (6, 700, 128), (6, 300, 44)])
def test_many_equals(dtype, W, equals, K):
    """More equals than are ranked by counting; totals near 0, where steps of float32 are far smaller than what the sums leave."""
    V = 20001
    near_zero = np.log(equals + (V - equals) * np.exp(0.5 - 12.0))
    check(480 // W, W, V, equals, 12.0, dtype, W + K, 0.2, K)
    check(480 // W, W, V, equals, 12.0, dtype, W + K, float(np.float32(near_zero)), K)


def test_the_same_logits_at_other_addresses():
    """Equal beams, whose rows begin at other places of a 16-byte word: every total is a tie, and the lower beam comes first."""
    x = torch.randn((1, 20001), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    x[0, 100] = x[0, 18000] = x[0, 14000] = 12.0
    rows = x.expand(8 * 60, 20001).contiguous().cuda()
    for K in (1, 2, 3, 6):
        _, picked, tokens = sv.beam_select(rows, torch.full((60, 8), -0.75, device="cuda"), K)
        beam, token = np.divmod(np.arange(K), 3)
        for i in range(60):
            assert picked[i].tolist() == (8 * i + beam).tolist() and tokens[i].tolist() == np.array([100, 14000, 18000])[token].tolist()
