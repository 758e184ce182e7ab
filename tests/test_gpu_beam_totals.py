"""How far sv_beam_select's totals are off: by at most 2^-19 before any second summation, and half a step of float32 (2^-24 of
the value); the float64 sums' own error is below 2^-40."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("high", [3.0, 9.0, 20.0, 25.0, 30.0, 33.0])
def test_a_total_is_off_by_little(dtype, high):
    """One logit far above those that the sums begin with, late in its row; totals next to 0 show the sums' whole error."""
    rows, V = 1024, 20000
    g = torch.Generator().manual_seed(int(high))
    x = torch.randn((rows, V), generator=g).to(dtype)
    x[torch.arange(rows), 10000 + torch.randint(0, 10000, (rows,), generator=g)] = (high + torch.rand(rows, generator=g)).to(dtype)
    got = sv.beam_select(x.cuda(), torch.zeros((rows, 1), device="cuda"), 1)[0].double().cpu().numpy()[:, 0]
    d = x.double()
    want = (d.max(1).values - torch.logsumexp(d, 1)).numpy()
    assert (np.abs(got - want) <= 2.0 ** -19 + 2.0 ** -24 * np.abs(want)).all()
