"""sv_sample_rows with so many logits (64 MB and more) that rows with a top-k or min-p go by the maxima of 128-byte groups:
bit for bit the documented arithmetic, and what the same rows give in smaller calls."""
import math
import os
import sys

import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_sample import _gpu, defined, params, rows  # noqa: E402, F401

pytestmark = pytest.mark.gpu
BYTES = 64 << 20


def many(V, dtype):
    return -(-BYTES // (V * (2 if dtype == torch.bfloat16 else 4)))


def uniforms(R, M, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(1 << 24, (R, M), device="cuda", generator=g) / 2.0 ** 24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", ["k", "q", "kp", "kq", "pq", "kpq"])
@pytest.mark.parametrize("kind", ["normal", "ties", "zeros", "wide", "masked"])
def test_bit_exact(which, kind, dtype):
    V = 50021
    R = many(V, dtype)
    x, u = rows(kind, R, V, dtype, len(which) + len(kind)), uniforms(R, 2, 1)
    T, k, p, q = params(R, 3, which)
    ws = sv.sample_workspace(R, V)
    tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True, ws=ws)
    a, b, c = defined(x, T, u, k, p, q)
    assert torch.equal(cut, c) and torch.equal(tok, a) and torch.equal(prob, b)
    assert sv.sv_query_status(ws) == (sv.SV_OK, 0)


@pytest.mark.parametrize("V", [100, 129, 1024, 4095, 262144])
def test_sizes(V):
    for dtype in (torch.bfloat16, torch.float32):
        R = many(V, dtype)
        x, u = rows("normal", R, V, dtype, V), uniforms(R, 1, V)
        T, k, p, q = params(R, V, "kpq")
        tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True)
        a, b, c = defined(x, T, u, k, p, q)
        assert torch.equal(cut, c) and torch.equal(tok, a) and torch.equal(prob, b)
        del x, u, cut, c


@pytest.mark.parametrize("dtype,lead", [(torch.bfloat16, 1), (torch.bfloat16, 5), (torch.float32, 1), (torch.float32, 3)])
def test_strided_rows_at_any_alignment(dtype, lead):
    V, stride = 50021, 50033
    R = many(V, dtype)
    base = rows("normal", R + 1, stride, dtype, lead)
    x = base.flatten()[lead:lead + R * stride].view(R, stride)[:, :V]
    out = torch.full_like(base, 7.0)
    cut = out.flatten()[lead + 1:lead + 1 + R * stride].view(R, stride)[:, :V]
    T, k, p, q = params(R, 5, "kpq")
    u = uniforms(R, 1, 2)
    tok, prob, _ = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=cut)
    a, b, c = defined(x.contiguous(), T, u, k, p, q)
    assert torch.equal(cut, c) and torch.equal(tok, a) and torch.equal(prob, b)
    # nothing is written between the rows
    assert bool((out.flatten()[lead + 1:lead + 1 + R * stride].view(R, stride)[:, V:] == 7.0).all())
    # in place: the same, the other way
    y = base.clone()
    z = y.flatten()[lead:lead + R * stride].view(R, stride)[:, :V]
    tok, prob, _ = sv.sample(z, T, u, top_k=k, top_p=p, min_p=q, filtered=z)
    assert torch.equal(z, c) and torch.equal(tok, a) and torch.equal(prob, b)


def test_bad_rows_are_flagged_and_others_stand():
    V = 50021
    R = many(V, torch.float32)
    x, u = rows("normal", R, V, torch.float32, 4), uniforms(R, 2, 3)
    T, k, p, q = params(R, 9, "kpq")
    good = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True)
    x[3, 77], x[5, V - 1], x[8, 0] = math.nan, math.inf, math.nan
    x[11] = -math.inf
    T[20], k[22], p[24], q[26], u[28, 1] = -1.0, -3, 0.0, 1.5, 1.0
    ws = sv.sample_workspace(R, V)
    tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True, ws=ws)
    bad = [3, 5, 8, 20, 22, 24, 26, 28]
    others = [r for r in range(R) if r not in bad + [11]]
    assert bool((tok[bad] == -1).all()) and bool(prob[bad].isnan().all()) and bool((cut[bad] == -math.inf).all())
    assert bool((tok[11] == -1).all()) and bool((prob[11] == 0).all()) and bool((cut[11] == -math.inf).all())
    for a, b in zip((tok, prob, cut), good):
        assert torch.equal(a[others], b[others])
    assert sv.sv_query_status(ws)[1] == sv.SV_DEV_BAD_LOGIT | sv.SV_DEV_BAD_TEMPERATURE | sv.SV_DEV_BAD_FILTER


def test_the_same_in_smaller_calls_and_again():
    V = 50021
    R = many(V, torch.bfloat16)
    x, u = rows("normal", R, V, torch.bfloat16, 6), uniforms(R, 1, 5)
    T, k, p, q = params(R, 11, "kpq")
    ws = sv.sample_workspace(R, V)
    first = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True, ws=ws)
    again = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True, ws=ws)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    for i in range(0, R, 100):
        s = slice(i, i + 100)
        part = sv.sample(x[s], T[s], u[s], top_k=k[s], top_p=p[s], min_p=q[s], filtered=True)
        for a, b in zip(first, part):
            assert torch.equal(a[s], b)


# ---- 64 rows (clusters of four), some with top-p and no top-k -------------------------------------------------------
@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 151936), (torch.float32, 50021)])
@pytest.mark.parametrize("kind", ["normal", "ties", "wide", "masked"])
@pytest.mark.parametrize("apart", [0, 1, 10, 38, 39, 64])
def test_rows_apart(apart, kind, dtype, V):
    R = 64
    x, u = rows(kind, R, V, dtype, apart), uniforms(R, 3, 4)
    T, k, p, q = params(R, 13, "kpq")
    T = torch.where(T == 0, 0.8, T)
    k = torch.where(k == 0, 20, k.clamp(max=1000)).to(torch.int32)
    where = torch.randperm(R, generator=torch.Generator().manual_seed(apart))[:apart].cuda()
    k[where] = 0
    p[where] = torch.where(p[where] >= 1, 0.95, p[where])
    ws = sv.sample_workspace(R, V)
    for _ in range(2):
        tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True, ws=ws)
        a, b, c = defined(x, T, u, k, p, q)
        assert torch.equal(cut, c) and torch.equal(tok, a) and torch.equal(prob, b)
    assert sv.sv_query_status(ws) == (sv.SV_OK, 0)


def test_bad_rows_apart():
    R, V = 64, 50021
    x, u = rows("normal", R, V, torch.float32, 8), uniforms(R, 1, 6)
    T, k, p, q = (torch.full((R,), 0.9, device="cuda"), torch.full((R,), 30, dtype=torch.int32, device="cuda"),
                  torch.full((R,), 0.9, device="cuda"), torch.zeros(R, device="cuda"))
    k[::5] = 0
    good = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True)
    x[5, 3], x[10, 3], x[6, 4] = math.nan, math.inf, math.nan
    p[15], u[20, 0], T[25], k[31] = 1.5, 1.0, math.inf, -1
    x[30] = -math.inf
    ws = sv.sample_workspace(R, V)
    tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True, ws=ws)
    bad = [5, 6, 10, 15, 20, 25, 31]
    others = [r for r in range(R) if r not in bad + [30]]
    assert bool((tok[bad + [30]] == -1).all()) and bool(prob[bad].isnan().all()) and bool((cut[bad + [30]] == -math.inf).all())
    for a, b in zip((tok, prob, cut), good):
        assert torch.equal(a[others], b[others])
    assert sv.sv_query_status(ws)[1] == sv.SV_DEV_BAD_LOGIT | sv.SV_DEV_BAD_TEMPERATURE | sv.SV_DEV_BAD_FILTER


def test_rows_apart_on_a_stream_and_in_a_graph():
    # the calls' own order: what fills the logits before, what reads the tokens after
    R, V = 64, 50021
    base, u = rows("normal", R, V, torch.float32, 9), uniforms(R, 1, 7)
    T, k, p, q = params(R, 17, "kpq")
    k[::6], p[::6] = 0, 0.9
    ws = sv.sample_workspace(R, V)
    x = torch.empty_like(base)
    out = (torch.empty(R, 1, dtype=torch.int32, device="cuda"), torch.empty(R, 1, device="cuda"))
    after = torch.empty_like(out[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(scale):
        torch.mul(base, scale, out=x)
        sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, out=out, ws=ws)
        after.copy_(out[0])

    with torch.cuda.stream(side):
        for i in range(20):
            step(1.0 + i)
            a = defined(base * (1.0 + i), T, u, k, p, q)[0]
            assert torch.equal(after, a)
    graph = torch.cuda.CUDAGraph()
    scale = torch.ones((), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(3):
            step(scale)
    for i in range(5):
        scale.fill_(1.0 + i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(after, defined(base * (1.0 + i), T, u, k, p, q)[0])
