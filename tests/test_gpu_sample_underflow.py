"""sv_sample_rows where exponents underflow: logits so close together, at a temperature so high, that (x - max) log2(e) / T
rounds to -0, which reaches min-p's threshold of q = 1.  Bit for bit the documented arithmetic, by clusters and by maxima."""
import os
import sys

import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_sample import _gpu, defined  # noqa: E402, F401

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale,T", [(1e-40, 1e20), (1e-30, 1e20), (1e-25, 1e20), (1e-8, 3e38), (1.0, 3e38), (1e-40, 0.5)])
@pytest.mark.parametrize("many", [False, True])
def test_min_p_of_one(scale, T, dtype, many):
    V = 20011
    R = -(-(64 << 20) // (V * (2 if dtype == torch.bfloat16 else 4))) if many else 12
    g = torch.Generator(device="cuda").manual_seed(R)
    x = (torch.randn((R, V), generator=g, device="cuda") * scale).to(dtype)
    x[3::7, ::2] = -float("inf")
    u = torch.randint(1 << 24, (R, 2), device="cuda", generator=g) / 2.0 ** 24
    T = torch.full((R,), T, device="cuda")
    q = torch.ones(R, device="cuda")
    q[5::6] = 0.5
    for k in (None, V - 1, 1025, 50, 1):
        for p in (None, 0.9):
            kk = None if k is None else torch.full((R,), k, dtype=I32, device="cuda")
            pp = None if p is None else torch.full((R,), p, device="cuda")
            tok, prob, cut = sv.sample(x, T, u, top_k=kk, top_p=pp, min_p=q, filtered=True)
            a, b, c = defined(x, T, u, kk, pp, q)
            assert torch.equal(cut, c) and torch.equal(tok, a) and torch.equal(prob, b), (k, p)
