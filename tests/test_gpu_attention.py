"""sv_tree_attention on the GPU against the float64 oracle.

Bounds.  Products of bf16 are exact in float32.  out: the softmax weights that multiply v are rounded to
bf16 (each off by at most 2^-9 of itself, so the weighted mean by at most 2^-9 max|v|) and the result is rounded to bf16
(2^-9 |o| <= 2^-9 max|v|): 2^-8 max|v| together, and float32 sums of a few thousand terms add below 1 percent of
it.  lse: a dot product's float32 sum is off by at most D 2^-24 sum|q k|; 2^y and log add a few 2^-22 of the sum."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from oracle.attention import tree_attention
from synth.trees import tree_shape

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


TREES = {"one": [-1], "none": [], "chain": list(tree_shape([1] * 16, 17)), "mixed": list(tree_shape([3, 2, 1, 1], 16)),
         "wide": list(tree_shape([7, 1], 15)), "big": list(tree_shape([4, 3, 3, 2], 77)),
         "deep": list(tree_shape([2] + [1] * 80, 150))}


def case(lens, trees, Hq, Hk, D, ps, layout="slots", seed=0, stale="nan", layers=1):
    """Inputs whose unused slots hold NaN (or large values): (cache, tensors, numpy twins)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    parents = [TREES[t] for t in trees]
    counts = [len(p) for p in parents]
    offs = np.concatenate([[0], np.cumsum(counts)])
    held = [-(-(n + c) // ps) for n, c in zip(lens, counts)]
    pages = sum(held) + 3
    shape = (layers, pages, ps, Hk, D) if layout == "slots" else (layers, pages, Hk, ps, D)
    k, v = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    if layout == "heads":
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    order = torch.randperm(pages, generator=g, device="cuda").cpu().numpy()
    table = np.full((len(lens), max(held + [1])), -1)
    used = np.zeros((pages, ps), bool)
    at = 0
    for i, n in enumerate(held):
        table[i, :n] = order[at:at + n]
        at += n
        for s in range(lens[i] + counts[i]):
            used[table[i, s // ps], s % ps] = True
    unused = torch.tensor(~used, device="cuda")
    for t in (k, v):
        for layer in range(layers):
            t[layer][unused] = float("nan") if stale == "nan" else 3e38
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[torch.tensor(order[:at].copy(), device="cuda")] = 1
    cache = sv.PagedCache(k, v, refs, i32(table))
    q = (torch.randn((int(offs[-1]), Hq, D), generator=g, device="cuda") * 2).to(torch.bfloat16)
    parent = i32([x for p in parents for x in p])
    return dict(cache=cache, q=q, lens=i32(lens), offs=i32(offs), parent=parent, nmax=max(counts + [1]), table=table, held=held)


def check(c, layer=0, window=0, sinks=0, parent="given", scale=None, **kw):
    q, cache = c["q"], c["cache"]
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    par = c["parent"] if isinstance(parent, str) else parent
    out, lse = sv.tree_attention(q, cache, layer, c["lens"], c["offs"], par, c["nmax"], scale=scale, window=window, sinks=sinks, **kw)
    clean = lambda t: torch.nan_to_num(t[layer].double(), nan=0.0).clamp(-1e3, 1e3).cpu().numpy()  # noqa: E731
    k, v = clean(cache.k), clean(cache.v)
    par_np = None if par is None else par.cpu().numpy()
    want, want_lse = tree_attention(q.double().cpu().numpy(), k, v, c["table"], c["lens"].cpu().numpy(),
                                    c["offs"].cpu().numpy(), par_np, scale, window, sinks)
    vmax = np.abs(v[np.abs(v) < 100]).max()
    qk = scale * np.abs(q.double().cpu().numpy()).sum(-1).max() * np.abs(k[np.abs(k) < 100]).max()
    assert np.abs(out.double().cpu().numpy() - want).max(initial=0) <= 2.0 ** -8 * 1.01 * vmax
    err = np.abs(lse.double().cpu().numpy() - want_lse).max(initial=0)
    assert err <= D * 2.0 ** -24 * qk + 2.0 ** -20, err
    return out, lse


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 111, 112, 113, 126, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("Hq,Hk,D,ps", [(8, 2, 128, 16), (4, 4, 64, 8), (10, 2, 64, 32), (16, 1, 128, 64), (3, 3, 128, 128),
                                        (8, 1, 64, 256)])
@pytest.mark.parametrize("tree", ["one", "mixed", "chain"])
def test_lengths_at_every_edge(Hq, Hk, D, ps, tree):
    c = case(EDGES, [tree] * len(EDGES), Hq, Hk, D, ps, seed=Hq)
    check(c)
    assert sv.sv_query_status(sv.attention_workspace(c["cache"], Hq))[0] == sv.SV_OK


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
    c = case([900, 400, 300], ["mixed", "one", "deep"], 4, 2, 128, 16, seed=3)
    cache, window, sinks = c["cache"], 50, 5
    for i, n in enumerate([900, 400, 300]):
        for s in range(sinks, n - window + 1):
            cache.k[0, c["table"][i, s // 16], s % 16] = float("nan")
            cache.v[0, c["table"][i, s // 16], s % 16] = float("inf")
    # whole pages out of sight need not be held at all
    cache.page_table[0, 2:50] = -1
    c["table"][0, 2:50] = 0
    ws = sv.attention_workspace(cache, 4)
    check(c, window=window, sinks=sinks, ws=ws)
    assert sv.sv_query_status(ws) == (sv.SV_OK, 0)


@pytest.mark.parametrize("layout", ["slots", "heads"])
def test_layouts_strides_and_layers(layout):
    c = case([200, 77], ["mixed", "wide"], 6, 3, 128, 32, layout=layout, layers=3, stale="large", seed=8)
    full = torch.randn((c["q"].shape[0], 9, 128 + 8), device="cuda").to(torch.bfloat16)
    full[:, 2:8, :128] = c["q"]
    c["q"] = full[:, 2:8, :128]
    room = torch.full((c["q"].shape[0], 7, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    for layer in range(3):
        out, _ = check(c, layer=layer, out=room[:, 1:7, 8:])
    assert torch.all(room[:, 0] == 5) and torch.all(room[:, :, :8] == 5)
    c["q"] = c["q"].contiguous()
    head_major = c["q"].transpose(0, 1).contiguous().transpose(0, 1)      # [heads, rows, dim] in memory
    a, b = check(c, layer=1), check(dict(c, q=head_major), layer=1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_chain_without_parents_and_scales():
    c = case([100, 5], ["chain", "chain"], 8, 2, 64, 16, seed=1)
    a, b = check(c, parent=None), check(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(c, scale=1e-3)
    check(c, scale=1.5)


def test_peaked_and_growing_scores():
    """Scores that rise along the sequence by hundreds: the running maximum moves at every tile."""
    c = case([1000, 640], ["mixed", "one"], 4, 1, 64, 16, seed=2, stale="large")
    cache = c["cache"]
    u = torch.sign(torch.randn(64, device="cuda"))
    for i, n in enumerate([1000, 640]):
        s = torch.arange(n, device="cuda")
        ramp = (s.float() / n * 4).round(decimals=2)
        cache.k[0, torch.tensor(c["table"][i], device="cuda")[s // 16], s % 16, 0] = (ramp[:, None] * u).to(torch.bfloat16)
    c["q"] = (u * 8).expand_as(c["q"]).to(torch.bfloat16).contiguous()
    check(c)
    c["q"] = -c["q"]
    check(c)


def test_many_heads_and_rows():
    """More rows a key/value head than one tile of 128 holds."""
    c = case([700, 130, 0], ["big", "deep", "chain"], 32, 2, 128, 64, seed=6)
    check(c)
    check(c, window=90, sinks=2)


def test_one_long_context_is_split_and_joined():
    """A few requests over 30k slots: every head's cache is shared out over many CTAs."""
    torch.manual_seed(0)
    D, Hk, ps, n = 128, 2, 128, 30011
    k, v = (torch.randn((1, 260, ps, Hk, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randperm(260, device="cuda").int()[:240].view(1, 240).contiguous()
    cache = sv.PagedCache(k, v, torch.ones(260, dtype=torch.int32, device="cuda"), table)
    for q_heads in (2, 16):
        q = torch.randn((3, q_heads, D), device="cuda").to(torch.bfloat16)
        out, lse = sv.tree_attention(q, cache, 0, i32([n]), i32([0, 3]), None, 3)
        s = torch.arange(n + 3, device="cuda")
        kk = k[0, table[0].long()[s // ps], s % ps].double()
        vv = v[0, table[0].long()[s // ps], s % ps].double()
        for c in range(3):
            for h in range(q_heads):
                x = kk[:n + 1 + c, h // (q_heads // Hk)] @ q[c, h].double() * D ** -0.5
                o = torch.softmax(x, 0) @ vv[:n + 1 + c, h // (q_heads // Hk)]
                assert (out[c, h].double() - o).abs().max() <= 2.0 ** -8 * 1.01 * 6
                assert abs(lse[c, h].item() - torch.logsumexp(x, 0).item()) <= 1e-4


def test_bad_requests_get_zeros_and_others_stand():
    lens, trees = [30, 40, 50, 60, 70], ["mixed"] * 5
    good = case(lens, trees, 4, 2, 64, 16, seed=9)
    q = good["q"]
    args = (good["offs"], good["parent"], good["nmax"])
    want, want_lse = sv.tree_attention(q, good["cache"], 0, good["lens"], *args)
    n = 16

    def flagged(i, bit, lens=good["lens"], offs=good["offs"], parent=good["parent"], nmax=good["nmax"]):
        ws = sv.attention_workspace(good["cache"], 4)
        out, lse = torch.full_like(want, 9.0), torch.full_like(want_lse, 9.0)
        for _ in range(2):     # a flagged call leaves the workspace usable
            sv.tree_attention(q, good["cache"], 0, lens, offs, parent, nmax, out=out, lse=lse, ws=ws)
            st, bits = sv.sv_query_status(ws)
            assert st == sv.SV_ERR_DEVICE_INPUT and bits == bit, (bits, bit)
        own = torch.zeros(80, dtype=torch.bool, device="cuda")
        own[n * i:n * i + n] = True
        assert torch.all(out[own] == 0) and torch.all(lse[own] == -float("inf"))
        assert torch.equal(out[~own], want[~own]) and torch.equal(lse[~own], want_lse[~own])
        sv.tree_attention(q, good["cache"], 0, good["lens"], *args, out=out, lse=lse, ws=ws)
        assert torch.equal(out, want) and sv.sv_query_status(ws) == (sv.SV_OK, 0)

    flagged(1, sv.SV_DEV_BAD_SEQ, lens=i32([30, -1, 50, 60, 70]))
    flagged(4, sv.SV_DEV_BAD_SEQ, lens=i32([30, 40, 50, 60, 10 ** 6]))
    p = good["parent"].clone()
    p[2 * n + 5] = 5
    flagged(2, sv.SV_DEV_BAD_PARENT, parent=p)
    p[2 * n + 5] = -1
    flagged(2, sv.SV_DEV_BAD_PARENT, parent=p)
    entry = good["cache"].page_table[3, 1].item()
    for bad in (-1, 10 ** 6):
        good["cache"].page_table[3, 1] = bad
        ws = sv.attention_workspace(good["cache"], 4)
        out, lse = sv.tree_attention(q, good["cache"], 0, good["lens"], *args, ws=ws)
        assert sv.sv_query_status(ws) == (sv.SV_ERR_DEVICE_INPUT, sv.SV_DEV_BAD_PAGE)
        assert torch.all(out[3 * n:4 * n] == 0) and torch.all(lse[3 * n:4 * n] == -float("inf"))
        assert torch.equal(out[:3 * n], want[:3 * n]) and torch.equal(out[4 * n:], want[4 * n:])
        good["cache"].page_table[3, 1] = entry
    # more nodes than announced
    ws = sv.attention_workspace(good["cache"], 4)
    out, _ = sv.tree_attention(q, good["cache"], 0, good["lens"], good["offs"], good["parent"], n - 1, ws=ws)
    assert torch.all(out == 0) and sv.sv_query_status(ws)[1] == sv.SV_DEV_BAD_NODES


def test_offsets_past_32_bits():
    pages, ps, Hk, D = 32769 + 16, 128, 8, 128
    k = torch.empty((1, pages, ps, Hk, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 32
    last = [pages - 1, pages - 4, pages - 2]
    for t in (k, v):
        t[0, last] = torch.randn((3, ps, Hk, D), device="cuda").to(torch.bfloat16)
    cache = sv.PagedCache(k, v, torch.ones(pages, dtype=torch.int32, device="cuda"), i32([last]))
    q = torch.randn((2, 16, D), device="cuda").to(torch.bfloat16)
    out, lse = sv.tree_attention(q, cache, 0, i32([330]), i32([0, 2]), None, 2)
    kk, vv = k[0, last].flatten(0, 1).double(), v[0, last].flatten(0, 1).double()
    for c in range(2):
        for h in range(16):
            x = kk[:331 + c, h // 2] @ q[c, h].double() * D ** -0.5
            assert (out[c, h].double() - torch.softmax(x, 0) @ vv[:331 + c, h // 2]).abs().max() <= 2.0 ** -8 * 6
            assert abs(lse[c, h].item() - torch.logsumexp(x, 0).item()) < 1e-4


def test_repeats_are_identical_and_graphs_replay():
    c = case([2000, 3, 517], ["mixed", "one", "wide"], 8, 2, 128, 64, seed=12)
    ws = sv.attention_workspace(c["cache"], 8)
    call = lambda **kw: sv.tree_attention(c["q"], c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"], **kw)  # noqa: E731
    want, want_lse = call(ws=ws)
    for _ in range(20):
        out, lse = call(ws=ws)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out, lse = call()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(ws=ws, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
