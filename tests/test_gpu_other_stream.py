"""Calls on a stream that is not the current one: what they return is not overwritten by work that is still pending on the
current stream, for which the same memory was used before."""
import os
import sys

import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_attention import _gpu, case  # noqa: E402, F401

pytestmark = pytest.mark.gpu
I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16
WAIT = 200_000_000  # cycles that the current stream is busy for: about a tenth of a second


def leave_pending(like):
    """Blocks of these sizes go back to the current stream's pool while a fill of them is still waiting there."""
    torch.cuda.synchronize()
    blocks = [torch.empty_like(t) for t in like for _ in range(3)]
    torch.cuda._sleep(WAIT)
    for b in blocks:
        b.fill_(7)


def flat(result):
    return [t for t in (result if isinstance(result, (tuple, list)) else [result]) if t is not None]


def both(call):
    """The call on the current stream, then on another one with fills pending: the same results."""
    want = [t.clone() for t in flat(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()  # no other free blocks: the pool's next ones of these sizes are the pending ones
    leave_pending(want)
    got = flat(call(side))
    side.synchronize()
    torch.cuda.synchronize()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_sample():
    x = torch.randn(300, 5000, device="cuda")
    T, u = torch.ones(300, device="cuda"), torch.rand(300, 2, device="cuda").clamp(max=0.999)
    ws = sv.sample_workspace(300, 5000)
    both(lambda s: sv.sample(x, T, u, filtered=True, ws=ws, stream=s))
    both(lambda s: sv.sample(x, T, u, filtered=True, stream=s))


def test_streams_by_their_handles():
    x, T = torch.randn(300, 5000, device="cuda"), torch.ones(300, device="cuda")
    u, ws = torch.rand(300, 2, device="cuda").clamp(max=0.999), sv.sample_workspace(300, 5000)
    both(lambda s: sv.sample(x, T, u, filtered=True, ws=ws, stream=None if s is None else s.cuda_stream))
    want = sv.sample(x, T, u, filtered=True)
    for stream in (0, torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream):
        for a, b in zip(sv.sample(x, T, u, filtered=True, stream=stream), want):
            assert torch.equal(a, b)


def test_attention():
    c = case([300, 700, 40], ["mixed", "chain", "one"], 8, 2, 128, 16)
    ws = sv.attention_workspace(c["cache"], 8)
    go = lambda s, **kw: sv.tree_attention(c["q"], c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"], stream=s, **kw)  # noqa: E731
    both(lambda s: go(s, ws=ws))
    both(lambda s: go(s))


def test_cache():
    cache = sv.PagedCache.empty(1, 4096, 8, 1, 64, 3000, 2)
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
    n = 1000
    lens, more = i32([3] * 3000), i32([2] * n)
    cache.reserve(lens, more)
    both(lambda s: cache.reserve(lens, more, stream=s))
    offs, path, acc = i32(range(0, 2 * n + 1, 2)), i32([[1, -1]] * n), i32([0, 1] * (n // 2))
    both(lambda s: cache.commit(lens, offs, path, acc, stream=s))
    src, dst = i32(range(n)), i32(range(n, 2 * n))
    both(lambda s: (cache.release(lens, dst, stream=s), cache.fork(lens, src, dst, stream=s))[1])


@pytest.mark.parametrize("own_ws", [True, False])
def test_verification(own_ws):
    B, K, V = 16, 4, 4000
    g = torch.Generator(device="cuda").manual_seed(0)
    t, d = (torch.randn(n, V, generator=g, device="cuda") for n in (B * (K + 1), B * K))
    tokens = torch.randint(V, (B, K), generator=g, device="cuda").to(I32)
    T = torch.ones(B, device="cuda")
    ws = sv.workspace(sv.SV_OP_VERIFY, B, K, V, sv.SV_F32) if own_ws else None
    both(lambda s: sv.verify_greedy(t, K, draft=d, ws=ws, stream=s))
    both(lambda s: sv.verify_sample(t, d, tokens, T, K, ws=ws, stream=s)[:2])
    keep = torch.full((B,), K, dtype=I32, device="cuda")
    row_t, row_d = (torch.arange(B + 1, dtype=I32, device="cuda") * n for n in (K + 1, K))
    both(lambda s: sv.verify_ragged(t, row_t, d, row_d, tokens, keep, T, K, ws=ws, stream=s)[:2])
    offs = torch.arange(B + 1, dtype=I32, device="cuda") * (K + 1)
    parent = torch.arange(-1, K, dtype=I32, device="cuda").repeat(B)
    drafted = torch.randint(V, (B * (K + 1),), generator=g, device="cuda").to(I32)
    rows = torch.randn(B * (K + 1), V, generator=g, device="cuda")
    tree = sv.workspace(sv.SV_OP_TREE, B, K + 1, V, sv.SV_F32) if own_ws else None
    both(lambda s: sv.verify_tree(t, rows, offs, parent, drafted, T, K + 1, ws=tree, stream=s)[2:])
    alpha = torch.rand(B, 8, generator=g, device="cuda")
    plan = sv.workspace(sv.SV_OP_SCHEDULE, B, 8, 1, sv.SV_F32) if own_ws else None
    both(lambda s: sv.schedule_depth(alpha, 1.0, 0.01, 40, ws=plan, stream=s))


def test_a_result_stays_while_the_current_stream_reads_it():
    """A result that the current stream still reads when it is dropped is not handed to the next call on the other stream."""
    x = torch.randn(400, 3000, device="cuda")
    T, u = torch.ones(400, device="cuda"), torch.rand(400, 2, device="cuda").clamp(max=0.999)
    ws = sv.sample_workspace(400, 3000)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    cut = sv.sample(x, T, u, top_k=torch.full((400,), 5, dtype=I32, device="cuda"), filtered=True, ws=ws, stream=side)[2]
    side.synchronize()
    want, copy = cut.clone(), torch.empty_like(cut)
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    copy.copy_(cut)
    del cut
    kept = [sv.sample(x, T, u, filtered=True, ws=ws, stream=side) for _ in range(6)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(kept) == 6
