"""sv_beam_select where a finished beam's score equals a live beam's total exactly: the lower beam comes first."""
import pytest
import torch

from test_gpu_beam import check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("finished", [[1, 0, 0, 0], [0, 1, 0, 0], [0, 0, 0, 1], [1, 0, 1, 0], [0, 1, 0, 1], [1, 1, 0, 0], [1, 1, 1, 1]])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 9])
def test_finished_beams_among_equals(dtype, finished, K):
    """A row with a single logit that is not -inf leaves its beam's score as it is."""
    x = torch.full((8, 700), -torch.inf)
    for w in range(8):
        x[w, 97 * w + 5] = float(w) - 3
    check(x.to(dtype), torch.full((2, 4), -2.25), K, torch.tensor([finished, finished[::-1]]), 3)


def test_one_token_in_all():
    check(torch.zeros((64, 1)), torch.full((1, 64), -7.0), 64, torch.arange(64)[None, :] % 2, 0)
    check(torch.zeros((64, 1)), torch.full((1, 64), -7.0), 40, (torch.arange(64)[None, :] + 1) % 2, 2 ** 30)
