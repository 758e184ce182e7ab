"""sample() of a single row: a row whose logits do not lie side by side is refused like several such rows are, and one row
gives what it gives among others."""
import os
import sys

import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16
V = 64


def go(logits, **kw):
    R = logits.shape[0]
    return sv.sample(logits, torch.ones(R), torch.zeros(R, 1), ws=torch.zeros(1 << 16, dtype=torch.uint8), **kw)


# views of R rows whose vocabulary dimension is not contiguous
APART = {"transposed": lambda R, dt: torch.zeros(V, 5, dtype=dt).t()[:R], "every second": lambda R, dt: torch.zeros(R, 2 * V, dtype=dt)[:, ::2],
         "one element": lambda R, dt: torch.zeros(1, dtype=dt).expand(R, V)}


@pytest.mark.parametrize("R", [1, 2])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("name", APART)
def test_rows_whose_logits_lie_apart_are_refused(name, dt, R):
    view, rows = APART[name](R, dt), torch.zeros(R, V, dtype=dt)
    with pytest.raises(ValueError, match="logit rows must be contiguous"):
        go(view)
    with pytest.raises(ValueError, match="logit rows must be contiguous"):
        go(rows, filtered=view)


def test_one_row_may_have_any_row_stride():
    # a CPU tensor that passes every other check stops at the device check
    for x in (torch.zeros(5, V)[2:3], torch.zeros(V).as_strided((1, V), (0, 1)), torch.zeros(V).as_strided((1, V), (1, 1)),
              torch.zeros(5, V)[::5], torch.zeros(3, 5)[:1, 2:3], torch.zeros(5, 3).t()[:1, 2:3]):
        with pytest.raises(ValueError, match="libsv takes device tensors"):
            go(x, filtered=torch.zeros(x.shape))
        with pytest.raises(ValueError, match="libsv takes device tensors"):
            go(torch.zeros(x.shape), filtered=x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [1, 7, 1000, 50021])
def test_one_row(vocab, dtype):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
    from test_gpu_sample import defined

    g = torch.Generator(device="cuda").manual_seed(vocab)
    base = (torch.randn((3, vocab + 3), generator=g, device="cuda") * 3).to(dtype)
    u = torch.randint(1 << 24, (1, 3), generator=g, device="cuda") / 2.0 ** 24
    T = torch.tensor([0.7], device="cuda")
    for filters in ({}, dict(top_k=torch.tensor([20], dtype=I32, device="cuda")), dict(top_p=torch.tensor([0.9], device="cuda")),
                    dict(top_k=torch.tensor([50], dtype=I32, device="cuda"), top_p=torch.tensor([0.8], device="cuda"),
                         min_p=torch.tensor([0.05], device="cuda"))):
        for x in (base[1:2, 1:1 + vocab], base[2, :vocab].as_strided((1, vocab), (0, 1))):
            a, b, c = defined(x, T, u, filters.get("top_k"), filters.get("top_p"), filters.get("min_p"))
            tok, prob, none = sv.sample(x, T, u, **filters)
            assert none is None and torch.equal(tok, a) and torch.equal(prob, b)
            room = torch.full((3, vocab + 5), 7.0, dtype=dtype, device="cuda")
            for cut in (True, room[1:2, 2:2 + vocab]):
                tok, prob, cut = sv.sample(x, T, u, filtered=cut, **filters)
                assert torch.equal(tok, a) and torch.equal(prob, b) and torch.equal(cut, c)
            room[1:2, 2:2 + vocab] = 7.0
            assert bool((room == 7.0).all())      # nothing beside the row was written
