"""sv_beam_select: totals beyond float32's range are the worst candidates, and do not push better ones out."""
import pytest
import torch

from test_gpu_beam import check, made

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("K", [8, 64, 128])
def test_the_lowest_number_beside_a_large_logit(K):
    x, scores = made(1, 6, 3000, torch.float32, K)
    x[:5] = LOWEST
    for w in range(5):
        x[w, 40 * w + 9] = 1e32 * (w + 1)
    # so many that all totals below are in float32's range: those of rows 0 to 4 but the first are not
    check(x, scores, K)


def test_scores_at_the_lowest_number():
    x, scores = made(1, 5, 2000, torch.float32, 1)
    scores[0, :4] = -3e38
    x[:4, 10:] = -1e38
    check(x, scores, 40)
