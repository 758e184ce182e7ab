"""sv_sample_rows where a row's finite logits lie further apart than the largest float (and where most of them are the type's
lowest value, or as far below the others as that), bit for bit the documented arithmetic: few rows (clusters) and many (the
maxima of 128-byte groups)."""
import os
import sys

import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_sample import _gpu, defined, params  # noqa: E402, F401

pytestmark = pytest.mark.gpu
V = 50021


def rows(kind, R, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((R, V), generator=g, device="cuda") * 3
    pick = torch.rand((R, V), generator=g, device="cuda")
    if kind == "span":         # distinct logits over the whole range of the type
        x = (x * 0.4e38).clamp(-3.3e38, 3.3e38)
    elif kind == "far":        # ordinary logits between 2e38 and -2e38
        x[pick < 0.0005], x[pick > 0.9] = 2e38, -2e38
    elif kind == "few":        # fewer of the largest than most top-k's ask for
        x[pick < 0.0002], x[pick > 0.5] = 2e38, -2e38
    elif kind == "top":        # one of 2e38, the others of the lowest value
        x.fill_(torch.finfo(dtype).min)
        x[:, 777] = 2e38
    elif kind == "lowest":     # most tokens masked with the lowest value
        x[pick > 0.05] = torch.finfo(dtype).min
    elif kind == "stretches":  # whole 128-byte groups masked with it, and large logits beside
        x[:, 1000:] = torch.finfo(dtype).min
        x[:, :400] *= 1e37
    return x.to(dtype)


def check(kind, R, dtype, which, seed):
    x = rows(kind, R, dtype, seed)
    assert bool(torch.isfinite(x.float()).all())
    T, k, p, q = params(R, seed, which)
    u = torch.randint(1 << 24, (R, 2), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) / 2.0 ** 24
    ws = sv.sample_workspace(R, V)
    tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True, ws=ws)
    a, b, c = defined(x, T, u, k, p, q)
    assert torch.equal(cut, c) and torch.equal(tok, a) and torch.equal(prob, b)
    assert sv.sv_query_status(ws) == (sv.SV_OK, 0)


KINDS = ["span", "far", "few", "top", "lowest", "stretches"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", ["", "k", "p", "q", "kp", "kq", "pq", "kpq"])
@pytest.mark.parametrize("kind", KINDS)
def test_few_rows(kind, which, dtype):
    check(kind, 24, dtype, which, len(which) + 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", ["k", "q", "kp", "kpq"])
@pytest.mark.parametrize("kind", KINDS)
def test_many_rows(kind, which, dtype):
    check(kind, -(-(64 << 20) // (V * (2 if dtype == torch.bfloat16 else 4))), dtype, which, 5)
