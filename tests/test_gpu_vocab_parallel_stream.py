"""Vocabulary-parallel verification on a stream that is not the current one, by a group of one rank (whose exchanges are
stand-ins: there is nobody to exchange with): its fills and steps are one sequence, whatever is pending on the current stream."""
import os
import sys

import pytest
import torch
import torch.distributed

import speculative_decoding_verification_74_gb300 as sv
from speculative_decoding_verification_74_gb300.dist import vocab_parallel_verify_sample

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_other_stream import _gpu, both  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def test_on_another_stream(monkeypatch):
    monkeypatch.setattr(torch.distributed, "get_rank", lambda group=None: 0)
    monkeypatch.setattr(torch.distributed, "get_world_size", lambda group=None: 1)
    monkeypatch.setattr(torch.distributed, "all_gather", lambda parts, local, group=None: parts[0].copy_(local))
    monkeypatch.setattr(torch.distributed, "all_reduce", lambda t, op=None, group=None: None)
    B, K, V = 12, 3, 20000
    g = torch.Generator(device="cuda").manual_seed(1)
    t, d = (torch.randn(n, V, generator=g, device="cuda") for n in (B * (K + 1), B * K))
    tokens = torch.randint(V, (B, K), generator=g, device="cuda").to(torch.int32)
    T = torch.ones(B, device="cuda")
    ws = sv.workspace(sv.SV_OP_VERIFY, B, K, V, sv.SV_F32)
    # p and q past the accepted length are not written
    both(lambda s: [vocab_parallel_verify_sample(t, d, tokens, T, K, V, seed=5, ws=ws, stream=s)[i] for i in (0, 1, 4)])
