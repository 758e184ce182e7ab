"""Workloads of the decoding-round operators around verification: sampling the drafter's (or the
target's) rows, attention of a token tree over a paged cache, and the cache's pages.

A case names its operator in "op":
  attend  sv.tree_attention: the nodes of a token tree against a paged key/value cache
  sample  sv.sample: draws from logit rows with temperature, top-k, top-p and min-p, and, with
          filtered, the rows with everything that cannot be drawn set to -inf
  turn    a cache's share of one round: PagedCache.reserve, append and commit
  fork    PagedCache.release and fork: beams that share pages

With `own` false, run() computes the same results with elementary torch operations.
"""
import math

import torch

own = False

LOG2E = 1.4426950408889634
FRACTION = 40          # fractional bits of a sampling weight
# Branching factors per level, as in this repository's tree workload: blocks of up to 16 nodes.
MIXED = "3-2-1-1-1/2-2-2-1/4-1-1-1-1-1/1-1-1-1-1-1-1-1-1-1-1-1-1-1-1/2-2-2-2/3-3-1/1-4-1-1/5-1-1"
CHAIN = "1-1-1-1-1-1-1-1-1-1-1-1-1-1-1-1"


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # four requests, one token each, short contexts: the latency of a call
        dict(name="attend_decode_b4", op="attend", requests=4, nodes=1, tree="", shortest=1, longest=130, q_heads=32,
             kv_heads=8, head_dim=128, page_size=16, window=0, sinks=0),
        # ordinary decoding at concurrency 64: one token per request, contexts of 6k to 8k
        dict(name="attend_decode_b64", op="attend", requests=64, nodes=1, tree="", shortest=6000, longest=8192,
             q_heads=32, kv_heads=8, head_dim=128, page_size=64, window=0, sinks=0),
        # the target's pass over the tree workload: 64 trees of up to 16 nodes in 8 shapes
        dict(name="attend_tree_b64", op="attend", requests=64, nodes=16, tree=MIXED, shortest=512, longest=4096,
             q_heads=32, kv_heads=8, head_dim=128, page_size=64, window=0, sinks=0),
        # a drafted block of 16 behind its root (a chain) over contexts of about 128k, few requests
        dict(name="attend_chain_long", op="attend", requests=4, nodes=17, tree=CHAIN, shortest=99001, longest=131072,
             q_heads=32, kv_heads=8, head_dim=128, page_size=128, window=0, sinks=0),
        # a drafter with a sliding window and four sinks, one key/value head per query head
        dict(name="attend_window_d64", op="attend", requests=33, nodes=16, tree=MIXED, shortest=1, longest=6000,
             q_heads=16, kv_heads=16, head_dim=64, page_size=32, window=1024, sinks=4),
        # four rows of the smallest vocabulary, plain temperature, float32: the latency of a call
        dict(name="sample_b4_f32", op="sample", rows=4, vocab=32000, stride=32001, dtype="f32", draws=1, top_k=False,
             top_p=False, min_p=False, filtered=False),
        # drafting a tree's first level at concurrency 64: three candidates a row, every filter, mixed parameters
        dict(name="sample_b64_filters", op="sample", rows=64, vocab=151936, stride=151936, dtype="bf16", draws=3,
             top_k=True, top_p=True, min_p=True, filtered=False),
        # cutting the target's rows of 64 requests with a block of 16 to their top-p sets before verification
        dict(name="sample_rows_cut", op="sample", rows=1088, vocab=151936, stride=151936, dtype="f32", draws=1,
             top_k=True, top_p=True, min_p=True, filtered=True),
        # one round of a small drafter's cache: latency
        dict(name="turn_b4", op="turn", requests=4, nodes=16, tree=MIXED, shortest=1, longest=130, layers=2,
             kv_heads=8, head_dim=128, page_size=16),
        # one round of a target's cache of 32 layers at concurrency 64
        dict(name="turn_b64", op="turn", requests=64, nodes=16, tree=MIXED, shortest=20, longest=100, layers=32,
             kv_heads=8, head_dim=128, page_size=64),
        # one prompt into three beams
        dict(name="fork_1_to_3", op="fork", requests=1, beams=3, shortest=37, longest=37, layers=2, kv_heads=8,
             head_dim=128, page_size=16),
        # sixteen prompts into 48 further beams, 32 layers: the copies of the partly filled pages
        dict(name="fork_16_to_48", op="fork", requests=16, beams=48, shortest=100, longest=300, layers=32, kv_heads=8,
             head_dim=128, page_size=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "sample", "sample", "turn", "fork"])
    if op == "attend":
        q_heads, kv_heads = rng.choice([(32, 8), (16, 16), (8, 1), (24, 8), (64, 8), (10, 2)])
        head_dim = rng.choice([64, 128])
        tree = rng.choice(["", MIXED, CHAIN, "4-3-2", "2-2-2-2-2"])
        nodes = 1 if tree == "" else rng.randint(2, 32)
        requests = _log(rng, 1, 64)
        longest = _log(rng, 1, max(1, min(131072, 500000 // (requests * (1 if kv_heads <= 8 else 2)))))
        shortest = rng.randint(0, longest)
        windowed = rng.random() < 0.3
        return dict(op=op, requests=requests, nodes=nodes, tree=tree, shortest=shortest, longest=longest,
                    q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page_size=rng.choice([16, 32, 64, 128]),
                    window=_log(rng, 1, 4096) if windowed else 0, sinks=rng.randint(0, 8) if windowed else 0)
    if op == "sample":
        vocab = _log(rng, 1000, 200000)
        rows = _log(rng, 1, max(1, min(1088, 165000000 // vocab)))
        return dict(op=op, rows=rows, vocab=vocab, stride=vocab + rng.randint(0, 9), dtype=rng.choice(["bf16", "f32"]),
                    draws=rng.choice([1, 1, 2, 3, 5]), top_k=rng.random() < 0.5, top_p=rng.random() < 0.5,
                    min_p=rng.random() < 0.5, filtered=rng.random() < 0.3)
    layers = _log(rng, 1, 32)
    kv_heads, head_dim = rng.choice([1, 2, 8]), rng.choice([64, 128])
    page_size = rng.choice([16, 32, 64])
    longest = rng.randint(1, 4 * page_size)
    if op == "turn":
        return dict(op=op, requests=_log(rng, 1, 64), nodes=rng.randint(1, 32),
                    tree=rng.choice([MIXED, CHAIN, "4-3-2", "2-2-2-2-2"]), shortest=rng.randint(0, longest), longest=longest,
                    layers=layers, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size)
    requests = _log(rng, 1, 16)
    return dict(op=op, requests=requests, beams=_log(rng, 1, 48), shortest=rng.randint(0, longest), longest=longest,
                layers=layers, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size)


def _lengths(case):
    """Cached tokens of each request: spread over [shortest, longest] in a mixed order."""
    n, lo, hi = case["requests"], case["shortest"], case["longest"]
    if n == 1:
        return [hi]
    step = next(k for k in (37, 41, 43, 47, 1) if math.gcd(k, n) == 1)
    return [lo + (hi - lo) * (i * step % n) // (n - 1) for i in range(n)]


def _parents(case):
    """Parent arrays of the requests' trees: breadth-first, level l branching as the text says, cut at `nodes`."""
    shapes = []
    for text in case["tree"].split("/"):
        parent, level = [-1], [0]
        for b in [int(x) for x in text.split("-") if x]:
            following = []
            for node in level:
                for _ in range(b):
                    if len(parent) < case["nodes"]:
                        parent.append(node)
                        following.append(len(parent) - 1)
            level = following
        shapes.append(parent)
    return [shapes[i % len(shapes)] for i in range(case["requests"])]


def _paths(case):
    """An accepted path per request: towards the last node, cut to a length that varies, none for some."""
    paths = []
    for i, parent in enumerate(_parents(case)):
        node, path = len(parent) - 1, []
        while node > 0:
            path.append(node)
            node = parent[node]
        path.reverse()
        paths.append(path[:len(path) - i % 3] if i % 5 != 4 else [])
    return paths


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _pool(case, seed, layers, spare):
    """A cache whose requests' pages lie scattered in the pool: (k, v, page_refs, page_table, generator)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ps, lens = case["page_size"], _lengths(case)
    used = [-(-n // ps) for n in lens]
    extra = spare(used)
    pages = sum(used) + extra
    shape = (layers, pages, ps, case["kv_heads"], case["head_dim"])
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return k, v, pages, used, lens, torch.randperm(pages, generator=g, device="cuda"), g


def _tables(used, order, pages, rows, width):
    table = torch.full((rows, width), -1, dtype=torch.int32)
    order = order.cpu().to(torch.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[order[:at].long()] = 1
    return table.cuda(), refs.cuda()


def _nodes(case, s):
    parents = _parents(case)
    counts = [len(p) for p in parents]
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    s.update(rows=offsets[-1], nmax=max(counts),
             node_offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
             parent=torch.tensor([x for p in parents for x in p], dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    op = case["op"]
    s = {"op": op, "case": case}
    if op == "sample":
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows, vocab, dtype = case["rows"], case["vocab"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # rows between flat (as of chat) and peaked (as of code): N(0, 1.5 to 3.5) with a Zipf tail on every other row
        x = torch.randn((rows, case["stride"]), generator=g, device="cuda")
        x *= 1.5 + 2 * torch.rand((rows, 1), generator=g, device="cuda")
        rank = (torch.rand((rows, case["stride"]), generator=g, device="cuda") * vocab + 1).log_()
        x[::2] -= 2 * rank[::2]
        s["logits"] = x.to(dtype)[:, :vocab]
        pick = lambda values: torch.tensor(values, device="cuda")[torch.randint(  # noqa: E731
            len(values), (rows,), generator=g, device="cuda")]
        s["temperature"] = pick([1.0, 0.6, 0.8, 1.3] if rows < 8 else [1.0, 0.6, 0.8, 1.3, 0.0])
        s["top_k"] = pick([50, 20, 0, 200, 1000]).to(torch.int32) if case["top_k"] else None
        s["top_p"] = pick([0.95, 0.9, 0.8, 1.0]) if case["top_p"] else None
        s["min_p"] = pick([0.05, 0.0, 0.02]) if case["min_p"] else None
        s["uniforms"] = torch.randint(1 << 24, (rows, case["draws"]), generator=g, device="cuda") / float(1 << 24)
        s["filtered"] = torch.empty((rows, vocab), dtype=dtype, device="cuda") if case["filtered"] else None
        if own:
            import speculative_decoding_verification_74_gb300 as sv
            s["ws"] = sv.sample_workspace(rows, vocab)
        return s
    if op == "attend":
        nodes = max(len(p) for p in _parents(case))
        ps = case["page_size"]
        k, v, pages, _, lens, order, g = _pool(case, seed, 1, lambda used: case["requests"] * (-(-nodes // ps) + 1) + 3)
        _nodes(case, s)
        width = -(-(max(lens) + nodes) // ps)
        table, refs = _tables([-(-(n + len(p)) // ps) for n, p in zip(lens, _parents(case))], order, pages,
                              case["requests"], width)
        s["q"] = 2 * torch.randn((s["rows"], case["q_heads"], case["head_dim"]), generator=g, device="cuda",
                                 dtype=torch.bfloat16)
        s["scale"] = case["head_dim"] ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((s["rows"], case["q_heads"]), device="cuda")
    elif op == "turn":
        ps, layers = case["page_size"], case["layers"]
        k, v, pages, used, lens, order, g = _pool(
            case, seed, layers, lambda used: case["requests"] * (-(-case["nodes"] // ps) + 1))
        _nodes(case, s)
        table, refs = _tables(used, order, pages, case["requests"], -(-(max(lens) + case["nodes"]) // ps))
        shape = (layers, s["rows"], case["kv_heads"], case["head_dim"])
        s["k_new"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        s["v_new"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        paths = _paths(case)
        s["counts"] = s["node_offsets"].diff()
        s["path"] = torch.tensor([p + [-1] * (s["nmax"] - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        s["accept_len"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        s["new_len"] = torch.empty(case["requests"], dtype=torch.int32, device="cuda")
        s["ok"] = torch.empty(case["requests"], dtype=torch.int32, device="cuda")
    else:
        k, v, pages, used, lens, order, g = _pool(case, seed, case["layers"], lambda used: case["beams"] + 2)
        lens = lens + [0] * case["beams"]
        table, refs = _tables(used, order, pages, case["requests"] + case["beams"], max(used) + 1)
        s["src"] = torch.tensor([i % case["requests"] for i in range(case["beams"])], dtype=torch.int32, device="cuda")
        s["dst"] = torch.arange(case["requests"], case["requests"] + case["beams"], dtype=torch.int32, device="cuda")
        s["ok"] = torch.empty(case["beams"], dtype=torch.int32, device="cuda")
    s.update(k=k, v=v, page_refs=refs, page_table=table,
             seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if own:
        import speculative_decoding_verification_74_gb300 as sv
        s["cache"] = sv.PagedCache(k, v, refs, table)
        if op == "attend":
            s["ws"] = sv.attention_workspace(s["cache"], case["q_heads"])
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    if s["op"] == "attend":
        return _plain_attend(s)
    if s["op"] == "sample":
        return _plain_sample(s)
    if s["op"] == "turn":
        _plain_reserve(s)
        _plain_append(s)
        _plain_commit(s)
    else:
        _plain_release(s)
        _plain_fork(s)
    return _cache_state(s)


def _cache_state(s):
    # the caches' bits: data that is moved has to arrive as it was
    out = dict(k=s["k"].view(torch.int16), v=s["v"].view(torch.int16), page_refs=s["page_refs"],
               page_table=s["page_table"], ok=s["ok"])
    out["length"] = s["new_len"] if s["op"] == "turn" else s["seq_len"]
    return out


def _own(s):
    import speculative_decoding_verification_74_gb300 as sv
    if s["op"] == "attend":
        out, lse = sv.tree_attention(s["q"], s["cache"], 0, s["seq_len"], s["node_offsets"], s["parent"], s["nmax"],
                                     scale=s["scale"], window=s["case"]["window"], sinks=s["case"]["sinks"], out=s["out"],
                                     lse=s["lse"], ws=s["ws"])
        return dict(out=out, lse=lse)
    if s["op"] == "sample":
        tokens, probs, _ = sv.sample(s["logits"], s["temperature"], s["uniforms"], top_k=s["top_k"], top_p=s["top_p"],
                                     min_p=s["min_p"], filtered=s["filtered"], ws=s["ws"])
        out = dict(tokens=tokens, probs=probs)
        if s["filtered"] is not None:
            out["filtered"] = s["filtered"]
        return out
    cache = s["cache"]
    if s["op"] == "turn":
        cache.reserve(s["seq_len"], s["counts"], ok=s["ok"])
        cache.append(s["k_new"], s["v_new"], s["seq_len"], s["node_offsets"])
        cache.commit(s["seq_len"], s["node_offsets"], s["path"], s["accept_len"], out_len=s["new_len"])
    else:
        cache.release(s["seq_len"], s["dst"])
        cache.fork(s["seq_len"], s["src"], s["dst"], ok=s["ok"])
    return _cache_state(s)


# ---- attention ---------------------------------------------------------------------------

def _plain_attend(s):
    k, v, q = s["k"][0], s["v"][0], s["q"].float()
    ps, lens, table = k.shape[1], s["seq_len"].long(), s["page_table"].long()
    B, N, Hq, Hk, D = lens.numel(), s["nmax"], q.shape[1], k.shape[2], q.shape[2]
    S = table.shape[1] * ps
    offs = s["node_offsets"].long()
    count = offs.diff()
    node = torch.arange(N, device="cuda")
    slot = torch.arange(S, device="cuda")
    there = node < count[:, None]                                        # [B, N]
    at = (offs[:-1, None] + node).clamp(max=s["rows"] - 1)
    # ancestors and self: with P[c, parent(c)] = 1, the inverse of I - P counts the paths up
    up = s["parent"].long()[at].clamp(min=0)
    link = ((up[:, :, None] == node) & (there & (node > 0))[:, :, None]).float()
    eye = torch.eye(N, device="cuda").expand(B, N, N)
    family = torch.linalg.solve_triangular(eye - link, eye, upper=False) > 0.5   # [B, N, N]
    depth = family.sum(-1) - 1
    j = slot - lens[:, None]                                             # [B, S] node at a slot
    cached = j < 0
    jc = j.clamp(0, N - 1)
    seen = family.gather(2, jc[:, None, :].expand(B, N, S)) & ((j >= 0) & (j < count[:, None]))[:, None, :]
    seen = (seen | cached[:, None, :]) & there[:, :, None]
    if s["case"]["window"] > 0:
        where = torch.where(cached, slot.expand(B, S), lens[:, None] + depth.gather(1, jc))
        here = lens[:, None] + depth
        seen &= (where < s["case"]["sinks"])[:, None, :] | (where[:, None, :] > here[:, :, None] - s["case"]["window"])
    pages = table.clamp(min=0)[:, slot // ps]
    kk = k[pages, slot % ps].float().permute(0, 2, 3, 1)                 # [B, Hk, D, S]
    vv = v[pages, slot % ps].float().permute(0, 2, 1, 3)                 # [B, Hk, S, D]
    G = Hq // Hk
    qq = q[at].view(B, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, N * G, D)
    x = (qq @ kk) * s["scale"]
    x = x.view(B, Hk, N, G, S).masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    o = (e.view(B, Hk, N * G, S) @ vv).view(B, Hk, N, G, D) / z
    lse = (m + torch.log(z)).view(B, Hk, N, G)
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), count, output_size=s["rows"])
    c = torch.arange(s["rows"], device="cuda") - offs[b]
    return dict(out=o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)[b, c].to(torch.bfloat16),
                lse=lse.permute(0, 2, 1, 3).reshape(B, N, Hq)[b, c])


# ---- sampling ----------------------------------------------------------------------------

def _share(total, part24):
    """floor(total * part24 / 2^24) in whole numbers."""
    return (total >> 24) * part24 + (((total & 0xFFFFFF) * part24) >> 24)


def _plain_sample(s):
    x, T = s["logits"].float(), s["temperature"]
    R, V = x.shape
    greedy = T == 0
    steep = torch.div(torch.full_like(T, LOG2E), torch.where(greedy, torch.ones_like(T), T))
    top = x.amax(1, keepdim=True)
    y = torch.where(top == -math.inf, torch.full_like(x, -math.inf), (x - top) * steep[:, None])
    w = torch.round(torch.exp2(y) * float(1 << FRACTION)).long()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    place = torch.arange(V, device="cuda")
    k = torch.full((R,), V, device="cuda") if s["top_k"] is None else torch.where(s["top_k"] <= 0, V, s["top_k"].long())
    k = torch.where(greedy, 1, k)
    keep = place < k[:, None]
    ws = w.gather(1, order) * keep
    if s["top_p"] is not None:
        p = torch.where(greedy, torch.ones_like(T), s["top_p"])
        limit = _share(ws.sum(1), torch.round(p * float(1 << 24)).long()).clamp(min=1)
        keep &= (p >= 1)[:, None] | ((ws.cumsum(1) - ws) < limit[:, None])
    if s["min_p"] is not None:
        keep &= y.gather(1, order) >= torch.where(greedy, torch.zeros_like(T), torch.log2(s["min_p"]))[:, None]
    kept = torch.zeros_like(keep).scatter(1, order, keep)
    kept &= x > -math.inf
    run_sum = (w * kept).cumsum(1)
    total = run_sum[:, -1:]
    at = _share(total, (s["uniforms"] * float(1 << 24)).long())
    token = torch.searchsorted(run_sum, at, right=True)
    none = total == 0
    prob = w.gather(1, token.clamp(max=V - 1)).float() / total.clamp(min=1).float()
    out = dict(tokens=torch.where(none, -1, token).int(), probs=torch.where(none, torch.zeros_like(prob), prob))
    if s["filtered"] is not None:
        out["filtered"] = x.masked_fill(~kept, -math.inf).to(s["logits"].dtype)
    return out


# ---- the cache ---------------------------------------------------------------------------

def _need(s, length):
    return (length.long() + s["k"].shape[2] - 1) // s["k"].shape[2]


def _plain_reserve(s):
    table, refs = s["page_table"], s["page_refs"]
    entry = torch.arange(table.shape[1], device="cuda")
    want = (entry < _need(s, s["seq_len"] + s["counts"])[:, None]) & (table < 0)
    free = torch.nonzero(refs == 0).flatten()
    ok = (want.sum(1).cumsum(0) <= free.numel()) | ~want.any(1)
    want &= ok[:, None]
    rank = (want.flatten().cumsum(0) - 1).view(want.shape).clamp(0, max(0, free.numel() - 1))
    if free.numel():
        table.copy_(torch.where(want, free[rank].int(), table))
        refs[free[rank[want]]] = 1
    s["ok"].copy_(ok)


def _places(s, request, slot):
    ps = s["k"].shape[2]
    return s["page_table"].long()[request, slot // ps], slot % ps


def _plain_append(s):
    B = s["seq_len"].numel()
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), s["counts"].long(), output_size=s["rows"])
    c = torch.arange(s["rows"], device="cuda") - s["node_offsets"].long()[b]
    page, slot = _places(s, b, s["seq_len"].long()[b] + c)
    s["k"][:, page, slot] = s["k_new"]
    s["v"][:, page, slot] = s["v_new"]


def _plain_commit(s):
    lens, path = s["seq_len"].long(), s["path"].long()
    b, j = torch.nonzero(torch.arange(path.shape[1], device="cuda") < s["accept_len"][:, None], as_tuple=True)
    page, slot = _places(s, b, lens[b] + path[b, j])
    to_page, to_slot = _places(s, b, lens[b] + 1 + j)
    s["k"][:, to_page, to_slot] = s["k"][:, page, slot]
    s["v"][:, to_page, to_slot] = s["v"][:, page, slot]
    s["new_len"].copy_(lens + torch.where(s["accept_len"] >= 0, s["accept_len"] + 1, 0))
    table = s["page_table"]
    back = (torch.arange(table.shape[1], device="cuda") >= _need(s, s["new_len"])[:, None]) & (table >= 0)
    s["page_refs"].index_add_(0, table[back].long(), torch.full_like(table[back], -1))
    table.masked_fill_(back, -1)


def _plain_release(s):
    rows = s["page_table"][s["dst"].long()]
    held = rows[rows >= 0].long()
    s["page_refs"].index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    s["page_table"][s["dst"].long()] = -1
    s["seq_len"][s["dst"].long()] = 0


def _plain_fork(s):
    src, dst, table, refs = s["src"].long(), s["dst"].long(), s["page_table"], s["page_refs"]
    ps = s["k"].shape[2]
    lens = s["seq_len"].long()[src]
    full, part = lens // ps, lens % ps
    free = torch.nonzero(refs == 0).flatten()
    split = part > 0
    rank = split.long().cumsum(0)
    ok = (rank <= free.numel()) | ~split
    entry = torch.arange(table.shape[1], device="cuda")
    share = (entry < full[:, None]) & ok[:, None]
    rows = torch.where(share, table[src], -1)
    refs.index_add_(0, rows[share].long(), torch.ones_like(rows[share]))
    new = torch.nonzero(split & ok).flatten()
    page = free[rank[new] - 1]
    old = table[src[new], full[new]].long()
    rows[new, full[new]] = page.int()
    refs[page] = 1
    used = (torch.arange(ps, device="cuda") < part[new][:, None])[None, :, :, None, None]
    s["k"][:, page] = torch.where(used, s["k"][:, old], s["k"][:, page])
    s["v"][:, page] = torch.where(used, s["v"][:, old], s["v"][:, page])
    table[dst] = rows
    s["seq_len"][dst] = torch.where(ok, lens, 0).int()
    s["ok"].copy_(ok)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"] * (2 if case["dtype"] == "bf16" else 4)
        draws = case["rows"] * case["draws"]
        return {"bytes": n * (2 if case["filtered"] else 1) + 12 * draws, "flops": 4 * case["rows"] * case["vocab"]}
    token = case["kv_heads"] * case["head_dim"] * 2 * 2                  # a token's keys and values in one layer
    lens = _lengths(case)
    if case["op"] == "attend":
        slots = pairs = rows = 0
        for n, parent in zip(lens, _parents(case)):
            depth = []
            for c, p in enumerate(parent):
                depth.append(0 if c == 0 else depth[p] + 1)
            rows += len(parent)
            read = n
            for c, d in enumerate(depth):
                cached, near = n, d + 1
                if case["window"] > 0:
                    first = max(0, n + d - case["window"] + 1)           # the window's first position
                    cached = max(0, n - first) + min(case["sinks"], first, n)
                    # ancestors at positions n..n + d: those in the window, and those among the first `sinks`
                    near = sum(1 for t in range(d + 1) if n + t >= first or n + t < case["sinks"])
                    read = cached if c == 0 else read
                pairs += cached + near
            slots += read + len(parent)
        row = case["q_heads"] * case["head_dim"] * 2
        return {"bytes": slots * token + rows * (2 * row + 4 * case["q_heads"]),
                "flops": 4 * case["q_heads"] * case["head_dim"] * pairs}
    token *= case["layers"]
    if case["op"] == "turn":
        rows = sum(len(p) for p in _parents(case))
        moved = sum(1 for path in _paths(case) for j, node in enumerate(path) if node != j + 1)
        return {"bytes": 2 * token * (rows + moved), "flops": 0}
    part = [lens[i % case["requests"]] % case["page_size"] for i in range(case["beams"])]
    return {"bytes": 2 * token * sum(part) + 64 * case["beams"], "flops": 0}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] not in ("attend", "sample"):
        return None                                                      # moved bits and whole numbers
    s = prepare(case, seed)
    return _exact_attend(s) if case["op"] == "attend" else _exact_sample(s)


def _exact_attend(s):
    """Request by request, head group by head group, over the slots that a node's path can see."""
    case, k, v = s["case"], s["k"][0], s["v"][0]
    ps, G = k.shape[1], case["q_heads"] // case["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty((s["rows"], case["q_heads"]), dtype=torch.float64, device="cuda")
    lens, table = s["seq_len"].tolist(), s["page_table"].long()
    first = 0
    for i, parent in enumerate(_parents(case)):
        L, N = lens[i], len(parent)
        slots = torch.arange(L + N, device="cuda")
        keys = k[table[i, slots // ps], slots % ps].double()             # [S, Hk, D]
        values = v[table[i, slots // ps], slots % ps].double()
        see = torch.zeros((N, L + N), dtype=torch.bool)
        for c in range(N):
            line, a = [], c
            while a >= 0:
                line.append(a)
                a = parent[a]
            d = len(line) - 1
            positions = list(range(L, L + d + 1))                        # of the ancestors, root first
            see[c, :L] = True
            for a, p in zip(reversed(line), positions):
                see[c, L + a] = case["window"] <= 0 or p < case["sinks"] or p > L + d - case["window"]
            if case["window"] > 0:
                see[c, min(L, case["sinks"]):max(0, min(L, L + d - case["window"] + 1))] = False
        see = see.cuda()
        q = s["q"][first:first + N].double().view(N, case["kv_heads"], G, -1)
        x = torch.einsum("nhgd,shd->nhgs", q, keys) * s["scale"]
        x = torch.where(see[:, None, None, :], x, -math.inf)
        lse[first:first + N] = torch.logsumexp(x, -1).view(N, -1)
        out[first:first + N] = torch.einsum("nhgs,shd->nhgd", torch.softmax(x, -1), values).reshape(N, case["q_heads"], -1)
        first += N
    return dict(out=out, lse=lse)


def _exact_sample(s):
    """Row by row with real-valued weights; the tokens are whole numbers and have no 64-bit value."""
    x = s["logits"]
    R, V = x.shape
    probs = torch.zeros(s["uniforms"].shape, dtype=torch.float64, device="cuda")
    cut = torch.empty((R, V), dtype=torch.float64, device="cuda") if s["filtered"] is not None else None
    temps = s["temperature"].double().tolist()
    for r in range(R):
        row = x[r].double()
        if temps[r] == 0:
            keep = torch.zeros(V, dtype=torch.bool, device="cuda")
            keep[torch.argmax(row)] = True
            e = torch.softmax(row, 0)
        else:
            e = torch.softmax(row / temps[r], 0)
            big, order = torch.sort(row, descending=True, stable=True)
            e_sorted = e[order]
            keep_sorted = torch.ones(V, dtype=torch.bool, device="cuda")
            if s["top_k"] is not None and s["top_k"][r] > 0:
                keep_sorted[int(s["top_k"][r]):] = False
            if s["top_p"] is not None and s["top_p"][r] < 1:
                within = e_sorted * keep_sorted
                ahead = within.cumsum(0) - within
                keep_sorted &= ahead < s["top_p"][r].double() * within.sum()
                keep_sorted[0] = True
            if s["min_p"] is not None:
                keep_sorted &= e_sorted >= s["min_p"][r].double() * e_sorted[0]
            keep = torch.zeros_like(keep_sorted)
            keep[order] = keep_sorted
        e = e * keep / (e * keep).sum()
        token = torch.searchsorted(e.cumsum(0), s["uniforms"][r].double(), right=True).clamp(max=V - 1)
        probs[r] = e[token]
        if cut is not None:
            cut[r] = torch.where(keep, row, -math.inf)
    return dict(tokens=None, probs=probs, filtered=cut) if cut is not None else dict(tokens=None, probs=probs)
