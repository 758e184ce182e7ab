"""sv_tree_attention4 on the GPU against the float64 oracle on the values that the codes stand for.

Bounds.  A stored value times an element of q is exact in float32.  A score's float32 sum is off by at most
D 2^-24 sum|q k|, and so is lse, with 2^-20 for 2^y and log.  out: a softmax weight is off by twice the score's bound
and 2^-11 for its float16 or 2^-8 for its bf16 (half a step), relative to itself; the weights add up to 1 within that, so out
is off by twice their sum times max|v|, and half a step of bf16 (2^-8) of itself."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from oracle import quant
from oracle.attention import tree_attention
from synth.trees import tree_shape

pytestmark = pytest.mark.gpu
K_SCALE, V_SCALE = 0.5, 0.25


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


TREES = {"one": [-1], "none": [], "chain": list(tree_shape([1] * 16, 17)), "mixed": list(tree_shape([3, 2, 1, 1], 16)),
         "wide": list(tree_shape([7, 1], 15)), "big": list(tree_shape([4, 3, 3, 2], 77)),
         "deep": list(tree_shape([2] + [1] * 80, 150)), "longest": list(range(-1, 1023))}


def case(lens, trees, Hq, Hk, D, ps, seed=0, layers=1, stride=0):
    """Inputs made by append, in a pool whose other slots hold bytes of 0xFF: codes of -6 under scales that are NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    parents = [TREES[t] for t in trees]
    counts = [len(p) for p in parents]
    total = [n + c for n, c in zip(lens, counts)]
    offs = np.concatenate([[0], np.cumsum(counts)])
    held = [-(-n // ps) for n in total]
    pages = sum(held) + 3
    n = ps * 9 * D // 8
    pool = torch.full((layers, pages, Hk, n + stride), 255, dtype=torch.uint8, device="cuda")[..., :n]
    order = torch.randperm(pages, generator=g, device="cuda").cpu().numpy()
    table = np.full((len(lens), max(held + [1])), -1)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = order[at:at + h]
        at += h
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[torch.tensor(order[:at].copy(), device="cuda")] = 1
    cache = sv.PagedCache4(pool, refs, i32(table), ps, D, k_scale=K_SCALE, v_scale=V_SCALE)
    k, v = (torch.randn((layers, sum(total), Hk, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache.append(k, v, i32([0] * len(lens)), i32(np.concatenate([[0], np.cumsum(total)])))
    q = (torch.randn((int(offs[-1]), Hq, D), generator=g, device="cuda") * 2).to(torch.bfloat16)
    return dict(cache=cache, q=q, lens=i32(lens), offs=i32(offs), parent=i32([x for p in parents for x in p]),
                nmax=max(counts + [1]), table=table, counts=counts)


def check(c, layer=0, window=0, sinks=0, parent="given", scale=None, **kw):
    q, cache = c["q"], c["cache"]
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    par = c["parent"] if isinstance(parent, str) else parent
    out, lse = sv.tree_attention(q, cache, layer, c["lens"], c["offs"], par, c["nmax"], scale=scale, window=window, sinks=sinks, **kw)
    pool = cache.pool[layer].cpu().numpy()
    k, v = quant.read(pool, D, cache.page_size, K_SCALE, False), quant.read(pool, D, cache.page_size, V_SCALE, True)
    want, want_lse = tree_attention(q.double().cpu().numpy(), k, v, c["table"], c["lens"].cpu().numpy(),
                                    c["offs"].cpu().numpy(), None if par is None else par.cpu().numpy(), scale, window, sinks)
    if want.size:
        qk = scale * np.abs(q.double().cpu().numpy()).sum(-1).max() * np.abs(k).max()
        score = D * 2.0 ** -24 * qk
        assert np.abs(lse.double().cpu().numpy() - want_lse).max() <= score + 2.0 ** -20
        bound = 2 * (2 * score + 2.0 ** -8) * np.abs(v).max() + 2.0 ** -8 * np.abs(want)
        assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()
        # and on the whole as near as bf16 comes: roundings of weights average out
        off = np.linalg.norm(out.double().cpu().numpy() - want)
        assert off <= 2.0 ** -8 * np.linalg.norm(want)
    return out, lse


EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 111, 112, 113, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("Hq,Hk,D,ps", [(8, 2, 128, 16), (4, 4, 64, 8), (10, 2, 64, 32), (16, 1, 128, 64), (3, 3, 128, 128),
                                        (8, 1, 64, 256), (40, 1, 128, 8)])
@pytest.mark.parametrize("tree", ["one", "mixed", "chain"])
def test_lengths_at_every_edge(Hq, Hk, D, ps, tree):
    c = case(EDGES, [tree] * len(EDGES), Hq, Hk, D, ps, seed=Hq)
    ws = sv.attention_workspace(c["cache"], Hq)
    check(c, ws=ws)
    assert sv.sv_query_status(ws) == (sv.SV_OK, 0)


@pytest.mark.parametrize("D", [64, 128])
def test_mixed_trees_in_one_batch(D):
    names = ["one", "big", "none", "deep", "mixed", "wide", "chain", "none"]
    c = case([40, 0, 500, 3, 700, 129, 1, 0], names, 12, 3, D, 16, seed=4)
    check(c)
    check(c, window=20, sinks=3)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (5, 4), (64, 0), (100, 200), (128, 4), (129, 1), (10 ** 6, 0)])
@pytest.mark.parametrize("tree", ["one", "mixed", "deep"])
def test_windows_and_sinks(window, sinks, tree):
    lens = [0, 1, 3, 4, 5, 100, 127, 128, 129, 260, 513, 700]
    c = case(lens, [tree] * len(lens), 4, 2, 64, 16, seed=window)
    check(c, window=window, sinks=sinks)


def test_slots_outside_every_window_may_hold_anything():
    lens, window, sinks = [900, 400, 300], 50, 5
    c = case(lens, ["mixed", "one", "deep"], 4, 2, 128, 16, seed=3)
    cache = c["cache"]
    want = sv.tree_attention(c["q"], cache, 0, c["lens"], c["offs"], c["parent"], c["nmax"], window=window, sinks=sinks)[0]
    for i, n in enumerate(lens):
        for s in range(-(-sinks // 8) * 8, (n - window + 1) // 8 * 8, 8):     # whole groups of eight slots
            cache.pool[0, c["table"][i, s // 16], :, (s % 16) // 8 * 1152:(s % 16) // 8 * 1152 + 1152] = 255
    cache.page_table[0, 2:50] = -1                                            # pages out of sight need not be held
    ws = sv.attention_workspace(cache, 4)
    got = sv.tree_attention(c["q"], cache, 0, c["lens"], c["offs"], c["parent"], c["nmax"], window=window, sinks=sinks, ws=ws)[0]
    assert torch.equal(got, want) and sv.sv_query_status(ws) == (sv.SV_OK, 0)


def test_strides_and_layers():
    c = case([200, 77], ["mixed", "wide"], 6, 3, 128, 32, layers=3, stride=48, seed=8)
    full = torch.randn((c["q"].shape[0], 9, 128 + 8), device="cuda").to(torch.bfloat16)
    full[:, 2:8, :128] = c["q"]
    c["q"] = full[:, 2:8, :128]
    room = torch.full((c["q"].shape[0], 7, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    for layer in range(3):
        check(c, layer=layer, out=room[:, 1:7, 8:])
    assert torch.all(room[:, 0] == 5) and torch.all(room[:, :, :8] == 5)
    plain = dict(c, q=c["q"].contiguous())
    assert torch.equal(check(plain, layer=1)[0], check(c, layer=1)[0])
    check(plain, parent=None)                                                 # chains


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1.0, 3e3])
def test_queries_of_any_size(size):
    """Small queries give flat softmaxes, large ones steep ones; rows scale by powers of two, so nothing else changes."""
    c = case([70, 150], ["mixed", "one"], 4, 2, 128, 16, seed=11)
    c["q"] = (c["q"].float() * size * torch.exp2(torch.arange(c["q"].shape[0], device="cuda") % 7)[:, None, None]).to(torch.bfloat16)
    out, lse = check(c, scale=1e-2 if size > 1 else None)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_a_query_that_is_not_finite_gives_nan_alone():
    c = case([40, 9], ["mixed", "mixed"], 4, 2, 64, 8, seed=2)
    want, want_lse = check(c)
    q = c["q"].clone()
    q[3, 1, 7], q[20, 0, 0] = float("nan"), float("inf")
    out, lse = sv.tree_attention(q, c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"])
    assert torch.isnan(out[3, 1]).all() and torch.isnan(out[20, 0]).all()
    keep = torch.ones(want.shape[:2], dtype=torch.bool, device="cuda")
    keep[3, 1] = keep[20, 0] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])


def test_split_contexts_and_many_requests():
    """One context over all CTAs, and more row tiles than CTAs."""
    check(case([20000], ["one"], 2, 1, 128, 64, seed=1))
    check(case([9000, 3], ["big", "one"], 4, 1, 64, 32, seed=1))
    check(case([5 + 3 * i for i in range(100)], ["one"] * 100, 8, 4, 64, 16, seed=1))


def test_bad_requests_get_zeros_and_leave_the_others():
    c = case([40, 50, 60, 70], ["mixed"] * 4, 4, 2, 128, 16, seed=6)
    ws = sv.attention_workspace(c["cache"], 4)
    want = check(c, ws=ws)
    n = c["counts"][0]

    def run(status, bad, **over):
        a = {**dict(lens=c["lens"], offs=c["offs"], parent=c["parent"]), **over}
        out, lse = sv.tree_attention(c["q"], c["cache"], 0, a["lens"], a["offs"], a["parent"], c["nmax"], ws=ws)
        assert sv.sv_query_status(ws)[1] == status
        rows = torch.arange(4 * n, device="cuda") // n
        for i in range(4):
            if i in bad:
                assert (out[rows == i] == 0).all() and (lse[rows == i] == -torch.inf).all()
            else:
                assert torch.equal(out[rows == i], want[0][rows == i]) and torch.equal(lse[rows == i], want[1][rows == i])

    parent = c["parent"].clone()
    parent[2 * n + 5] = 9
    run(sv.SV_DEV_BAD_PARENT, [2], parent=parent)
    lens = c["lens"].clone()
    lens[1] = -1
    run(sv.SV_DEV_BAD_SEQ, [1], lens=lens)
    lens[1] = 10 ** 6
    run(sv.SV_DEV_BAD_SEQ, [1], lens=lens)
    table = c["cache"].page_table.clone()
    for page in (-1, 10 ** 6):
        c["cache"].page_table[3, 1] = page
        run(sv.SV_DEV_BAD_PAGE, [3])
    c["cache"].page_table.copy_(table)
    run(0, [])


def test_other_stream_and_replay():
    c = case([130, 260], ["mixed", "chain"], 8, 2, 128, 16, seed=9)
    want = check(c)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = sv.attention_workspace(c["cache"], 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.tree_attention(c["q"], c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.tree_attention(c["q"], c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"], out=out, lse=lse, ws=ws)
    for _ in range(3):
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("Hq,Hk", [(16, 4), (18, 3)])
def test_many_tiles_of_64_dimensions(Hq, Hk):
    """Pairs of heads and single ones, row tiles over many cache tiles."""
    check(case([5000, 2100, 900], ["mixed", "wide", "chain"], Hq, Hk, 64, 32, seed=Hq))


@pytest.mark.parametrize("D", [64, 128])
def test_more_requests_than_leave_room_for_four_stages(D):
    lens = [(37 * i) % 300 for i in range(1700)]
    c = case(lens, ["wide" if i % 8 == 0 else "one" for i in range(1700)], 4, 2, D, 16, seed=D)
    check(c)


def test_one_workspace_for_few_and_many_rows():
    few, many = case([300, 40], ["one", "one"], 8, 2, 128, 16, seed=1), case([300, 40], ["big", "mixed"], 8, 2, 128, 16, seed=2)
    ws = sv.attention_workspace(few["cache"], 8)
    for _ in range(2):
        check(few, ws=ws)
        check(many, ws=ws)


@pytest.mark.parametrize("tree", ["one", "mixed"])
def test_rows_behind_the_last_request_stay(tree):
    c = case([100, 30], [tree] * 2, 8, 2, 64, 16, seed=3)
    n = c["q"].shape[0]
    q = torch.cat([c["q"], torch.full((5, 8, 64), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out, lse = torch.full((n + 5, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((n + 5, 8), 9.0, device="cuda")
    parent = torch.cat([c["parent"], i32([-1] * 5)])
    sv.tree_attention(q, c["cache"], 0, c["lens"], c["offs"], parent, c["nmax"], out=out, lse=lse)
    want, want_lse = sv.tree_attention(c["q"], c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"])
    assert torch.equal(out[:n], want) and torch.equal(lse[:n], want_lse)
    assert (out[n:] == 7).all() and (lse[n:] == 9).all()


@pytest.mark.parametrize("tree", ["one", "mixed"])
def test_pages_past_four_gigabytes(tree):
    """The same sequences in a small pool and in pages whose bytes lie behind 2^32."""
    pages, ps, D, Hk = 60000, 64, 128, 8
    outs = []
    for count, first in ((40, 0), (pages, pages - 40)):
        table = i32([[first + 7, first + 30, first + 2, first + 39], [first + 11, first + 1, -1, -1], [-1] * 4])
        refs = torch.zeros(count, dtype=torch.int32, device="cuda")
        refs[table[table >= 0].long()] = 1
        refs[:first] = 1
        cache = sv.PagedCache4(torch.empty((1, count, Hk, ps * 9 * D // 8), dtype=torch.uint8, device="cuda"), refs, table, ps, D)
        g = torch.Generator(device="cuda").manual_seed(4)
        parent = TREES[tree]
        N = len(parent)
        k, v = (torch.randn((1, 330 + 2 * N, Hk, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        q = torch.randn((2 * N, 32, D), generator=g, device="cuda").to(torch.bfloat16)
        cache.append(k, v, i32([0, 0, 0]), i32([0, 230 + N, 330 + 2 * N, 330 + 2 * N]))
        args = (i32([0, N, 2 * N, 2 * N]), i32(parent * 2), N)
        lens = i32([230, 100, 0])
        one = sv.tree_attention(q, cache, 0, lens, *args)
        assert int(cache.reorder(lens, i32([1, 0, 0]))) == 1
        two = sv.tree_attention(q[:N], cache, 0, lens, i32([0, 0, 0, N]), i32(parent), N)  # the copied row, without its tree's slots
        outs.append((*one, lens))
        assert cache.page_table[2, 3] != cache.page_table[1, 3] and cache.page_table[2, 0] == cache.page_table[1, 0]
        assert two[0].shape == (N, 32, D)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
def test_the_longest_chain_and_the_most_requests(D):
    c = case([100, 5], ["longest", "one"], 4, 2, D, 64, seed=D)
    check(c)
    check(c, parent=None)
    check(c, window=700, sinks=3)
    c = case([i % 40 for i in range(4096)], ["wide" if i % 300 == 0 else "one" for i in range(4096)], 4, 2, D, 16, seed=D)
    check(c)
