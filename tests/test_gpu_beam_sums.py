"""sv_beam_select's sums of exponentials over logits far from 0, and masks of any large negative number.  Bounds as in
test_gpu_beam."""
import pytest
import torch

from test_gpu_beam import check, made

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("shift", [3e3, 5e3, -2e4, 1e5, -1e6, 2e7, -1e9, 4e9, -1e12, 1e20, -1e29, 3e30])
@pytest.mark.parametrize("V", [900, 20001])
def test_logits_far_from_zero(shift, V):
    """The differences are those that float32 leaves next to the shift."""
    x, scores = made(3, 3, V, torch.float32, 3)
    check(x + shift, scores, 12)
    check((x + shift).to(torch.bfloat16), scores, 12)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mask", [-5e3, -1e4, -1e6, -1e9, -1e10, -3e15, -1e25, -1e30, -3.38e38])
def test_masks_of_finite_numbers(dtype, mask):
    """Masks over the beginning, the end, most and all of a row."""
    x, scores = made(2, 4, 30000, dtype, 4)
    x[0, :20000] = mask
    x[1, 9000:] = mask
    x[2] = mask
    x[2, 29000:29040] = 1.5
    x[3] = mask
    x[4, ::2] = mask
    x[5, 17:] = mask
    x[6, :29999] = mask
    x[7, torch.arange(30000) % 4096 < 4000] = mask
    check(x, scores, 16)
