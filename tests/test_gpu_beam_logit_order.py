"""sv_beam_select: within a beam the order is that of the logits, also where float64 totals cannot tell them apart."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def order(x, K):
    return np.lexsort((np.arange(len(x)), -x.double().numpy()))[:K].tolist()


@pytest.mark.parametrize("V,K", [(100, 64), (100, 128), (5001, 128), (60000, 20)])
def test_small_differences(V, K):
    """Logits next to 0 that differ by far less than a step of the totals; some are equal."""
    x = torch.randint(0, 40, (V,), generator=torch.Generator().manual_seed(V)).float() * 1e-25
    x[V // 2] = 5.0
    _, rows, tokens = sv.beam_select(x[None, :].cuda(), torch.tensor([[-3.0]], device="cuda"), K)
    n = min(V, K)
    assert tokens[0, :n].tolist() == order(x, n) and (tokens[0, n:] == -1).all() and (rows[0, :n] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scores_that_swallow_the_logits(dtype):
    """Scores of -1e30: every candidate's total is the score, beams come one after the other, each in the order of its logits."""
    x = torch.randn((3, 4000), generator=torch.Generator().manual_seed(1)).to(dtype)
    _, rows, tokens = sv.beam_select(x.cuda(), torch.full((1, 3), -1e30, device="cuda"), 50)
    assert (rows == 0).all() and tokens[0].tolist() == order(x[0], 50)
    _, rows, tokens = sv.beam_select(x.cuda(), torch.full((1, 3), -1e30, device="cuda"), 50,
                                     finished=torch.tensor([[1, 0, 0]], dtype=torch.int32, device="cuda"), pad=9)
    assert rows[0].tolist() == [0] + [1] * 49 and tokens[0].tolist() == [9] + order(x[1], 49)
