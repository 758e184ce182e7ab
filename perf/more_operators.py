"""Workloads of the operators that a paged cache held in 4 bits and a beam search over it add to a
decoding round.

A case names its operator in "op":
  attend4  sv.tree_attention on a PagedCache4: a token tree's attention over keys and values of 4 bits
  turn4    a 4-bit cache's share of one round: PagedCache4.reserve, append (which quantises) and commit
  beam     sv.beam_select: the best continuations over all beams of a request and the vocabulary
  reorder  PagedCache.reorder (bits = 16) or PagedCache4.reorder (bits = 4): every sequence becomes a copy
           of the one that its beam goes on from

With `own` false, run() computes the same results with elementary torch operations.

The 4-bit format.  Sixteen neighbouring dimensions of a token's key (or value) in one head share a scale: with
t = x / (the cache's k_scale or v_scale, as a product with its float32 reciprocal), the scale is max|t| * (1/6)
rounded to e4m3 (at most 448), a code is t / scale rounded to e2m1 (sign and one of 0, .5, 1, 1.5, 2, 3, 4, 6; ties to
the even code, 6 at most; 0 where the scale is 0).  A head's page lies in groups of eight slots, 9 D bytes each:
  4 D    key codes, slot by slot; a byte holds an even dimension (low half) and the next one
  D / 2  key scales, slot by slot
  4 D    value codes: for each eighth of the dimensions, for each pair of slots, the even slot's and the odd slot's
  D / 2  value scales: for each sixteen dimensions, the eight slots'
Caches are returned as these bytes: codes and scales have to be equal.
"""
import math

import torch

own = False

# Branching factors per level, as in this repository's tree workload: blocks of up to 16 nodes.
MIXED = "3-2-1-1-1/2-2-2-1/4-1-1-1-1-1/1-1-1-1-1-1-1-1-1-1-1-1-1-1-1/2-2-2-2/3-3-1/1-4-1-1/5-1-1"
CHAIN = "1-1-1-1-1-1-1-1-1-1-1-1-1-1-1-1"
SIXTH = 1.0 / 6.0


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # four requests, one token each, short contexts: the latency of a call
        dict(name="attend4_decode_b4", op="attend4", requests=4, nodes=1, tree="", shortest=1, longest=130, q_heads=32,
             kv_heads=8, head_dim=128, page_size=16, window=0, sinks=0),
        # ordinary decoding at concurrency 64: one token per request, contexts of 6k to 8k
        dict(name="attend4_decode_b64", op="attend4", requests=64, nodes=1, tree="", shortest=6000, longest=8192,
             q_heads=32, kv_heads=8, head_dim=128, page_size=64, window=0, sinks=0),
        # the target's pass over the tree workload: 64 trees of up to 16 nodes in 8 shapes
        dict(name="attend4_tree_b64", op="attend4", requests=64, nodes=16, tree=MIXED, shortest=512, longest=4096,
             q_heads=32, kv_heads=8, head_dim=128, page_size=64, window=0, sinks=0),
        # a drafted block of 16 behind its root (a chain) over contexts of about 128k, few requests
        dict(name="attend4_chain_long", op="attend4", requests=4, nodes=17, tree=CHAIN, shortest=99001, longest=131072,
             q_heads=32, kv_heads=8, head_dim=128, page_size=128, window=0, sinks=0),
        # a drafter with a sliding window and four sinks, one key/value head per query head
        dict(name="attend4_window_d64", op="attend4", requests=33, nodes=16, tree=MIXED, shortest=1, longest=6000,
             q_heads=16, kv_heads=16, head_dim=64, page_size=32, window=1024, sinks=4),
        # one round of a small drafter's cache: latency
        dict(name="turn4_b4", op="turn4", requests=4, nodes=16, tree=MIXED, shortest=1, longest=130, layers=2,
             kv_heads=8, head_dim=128, page_size=16),
        # one round of a target's cache of 32 layers at concurrency 64
        dict(name="turn4_b64", op="turn4", requests=64, nodes=16, tree=MIXED, shortest=20, longest=100, layers=32,
             kv_heads=8, head_dim=128, page_size=64),
        # one request of four beams, the smallest vocabulary: the latency of a call
        dict(name="beam_b1_w4", op="beam", requests=1, beams=4, vocab=32000, stride=32001, dtype="bf16", candidates=8,
             finished=False),
        # sixteen requests of four beams, some of them finished, float32
        dict(name="beam_b16_w4_f32", op="beam", requests=16, beams=4, vocab=151936, stride=151936, dtype="f32",
             candidates=8, finished=True),
        # sixty-four requests of sixteen beams, two candidates for each
        dict(name="beam_b64_w16", op="beam", requests=64, beams=16, vocab=151936, stride=151936, dtype="bf16",
             candidates=32, finished=False),
        # one request's four beams in a small drafter's cache: latency
        dict(name="reorder_b1_w4", op="reorder", requests=1, beams=4, shortest=37, longest=130, layers=2, kv_heads=8,
             head_dim=128, page_size=16, bits=16),
        # sixteen requests of four beams in a target's cache of 32 layers, held in 4 bits
        dict(name="reorder_b16_w4", op="reorder", requests=16, beams=4, shortest=100, longest=600, layers=32, kv_heads=8,
             head_dim=128, page_size=64, bits=4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend4", "attend4", "attend4", "turn4", "beam", "beam", "reorder"])
    if op == "attend4":
        q_heads, kv_heads = rng.choice([(32, 8), (16, 16), (8, 1), (24, 8), (64, 8), (10, 2)])
        head_dim = rng.choice([64, 128])
        tree = rng.choice(["", MIXED, CHAIN, "4-3-2", "2-2-2-2-2"])
        nodes = 1 if tree == "" else rng.randint(2, 32)
        requests = _log(rng, 1, 64)
        longest = _log(rng, 1, max(1, min(131072, 500000 // (requests * (1 if kv_heads <= 8 else 2)))))
        shortest = rng.randint(0, longest)
        windowed = rng.random() < 0.3
        return dict(op=op, requests=requests, nodes=nodes, tree=tree, shortest=shortest, longest=longest,
                    q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page_size=rng.choice([8, 16, 32, 64, 128]),
                    window=_log(rng, 1, 4096) if windowed else 0, sinks=rng.randint(0, 8) if windowed else 0)
    if op == "beam":
        vocab = _log(rng, 1000, 200000)
        beams = _log(rng, 1, 32)
        requests = _log(rng, 1, max(1, min(64, 155000000 // (vocab * beams))))
        return dict(op=op, requests=requests, beams=beams, vocab=vocab, stride=vocab + rng.randint(0, 9),
                    dtype=rng.choice(["bf16", "f32"]) if requests * beams <= 512 else "bf16",
                    candidates=rng.choice([beams, 2 * beams, beams + 1]), finished=rng.random() < 0.4)
    layers = _log(rng, 1, 32)
    kv_heads, head_dim = rng.choice([1, 2, 8]), rng.choice([64, 128])
    page_size = rng.choice([16, 32, 64])
    longest = rng.randint(1, 4 * page_size)
    if op == "turn4":
        return dict(op=op, requests=_log(rng, 1, 64), nodes=rng.randint(1, 32),
                    tree=rng.choice([MIXED, CHAIN, "4-3-2", "2-2-2-2-2"]), shortest=rng.randint(0, longest), longest=longest,
                    layers=layers, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size)
    return dict(op=op, requests=_log(rng, 1, 16), beams=rng.randint(1, 4), shortest=rng.randint(0, longest), longest=longest,
                layers=layers, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size, bits=rng.choice([4, 16]))


def _lengths(case, n):
    """Cached tokens of n sequences: spread over [shortest, longest] in a mixed order."""
    lo, hi = case["shortest"], case["longest"]
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


def _sources(case):
    """The sequence that each beam goes on from: within its request, some twice or more, so some beams end."""
    W = case["beams"]
    return [i * W + [j, j // 2, 0, W - 1 - j, (j + 1) % W][i % 5] for i in range(case["requests"]) for j in range(W)]


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _tables(used, order, pages, width):
    table = torch.full((len(used), width), -1, dtype=torch.int32)
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


def _fill(case, pool, g, k_scale, v_scale):
    """A pool that holds quantised normal keys and values in every slot."""
    L, P, H, _ = pool.shape
    ps, D = case["page_size"], case["head_dim"]
    some = max(1, (1 << 26) // (H * ps * D))
    for layer in range(L):
        for p0 in range(0, P, some):
            part = pool[layer:layer + 1, p0:p0 + some]
            n = part.shape[1]
            page = torch.arange(n, device="cuda").repeat_interleave(ps)
            slot = torch.arange(ps, device="cuda").repeat(n)
            x = torch.randn((1, n * ps, H, D), generator=g, device="cuda")
            _write(part, D, page, slot, _quantise(x, k_scale), _quantise(x.roll(1, 1), v_scale))


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": op, "case": case}
    if op == "beam":
        B, W, V, dtype = case["requests"], case["beams"], case["vocab"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # rows between flat (as of chat) and peaked (as of code): N(0, 1.5 to 3.5) with a Zipf tail on every other row
        x = torch.randn((B * W, case["stride"]), generator=g, device="cuda")
        x *= 1.5 + 2 * torch.rand((B * W, 1), generator=g, device="cuda")
        rank = (torch.rand((B * W, case["stride"]), generator=g, device="cuda") * V + 1).log_()
        x[::2] -= 2 * rank[::2]
        s["logits"] = x.to(dtype)[:, :V]
        # beams of a search under way lie close together; every fourth request is at its start: one beam only
        s["scores"] = -20 - 4 * torch.rand((B, W), generator=g, device="cuda")
        s["scores"][3::4, 1:] = -math.inf
        s["finished"] = (torch.rand((B, W), generator=g, device="cuda") < 0.25).int() if case["finished"] else None
        s["pad"] = V // 2
        if own:
            import speculative_decoding_verification_74_gb300 as sv
            s["ws"] = sv.beam_workspace(B * W, V, case["candidates"])
        return s
    ps, H, D = case["page_size"], case["kv_heads"], case["head_dim"]
    bits, layers = case.get("bits", 4), case.get("layers", 1)
    rows = case["requests"] * case.get("beams", 1)
    lens = _lengths(case, rows)
    if op == "attend4":
        nodes = max(len(p) for p in _parents(case))
        used, spare = [-(-(n + len(p)) // ps) for n, p in zip(lens, _parents(case))], 3
        width = -(-(max(lens) + nodes) // ps)
    elif op == "turn4":
        used, spare = [-(-n // ps) for n in lens], rows * (-(-case["nodes"] // ps) + 1)
        width = -(-(max(lens) + case["nodes"]) // ps)
    else:
        used, spare = [-(-n // ps) for n in lens], rows + 2
        width = max(used) + 1
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=g, device="cuda")            # the pages lie scattered in the pool
    table, refs = _tables(used, order, pages, width)
    s.update(page_refs=refs, page_table=table, seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             k_scale=0.5, v_scale=0.25)
    if bits == 4:
        s["pool"] = torch.empty((layers, pages, H, ps * 9 * D // 8), dtype=torch.uint8, device="cuda")
        if op == "attend4":
            _fill(case, s["pool"], g, s["k_scale"], s["v_scale"])
        else:
            s["pool"].random_(0, 256, generator=g)                       # data that is moved as it is
    else:
        for name in ("k", "v"):
            s[name] = torch.randn((layers, pages, ps, H, D), generator=g, device="cuda", dtype=torch.bfloat16)
    if op == "attend4":
        _nodes(case, s)
        s["q"] = 2 * torch.randn((s["rows"], case["q_heads"], D), generator=g, device="cuda", dtype=torch.bfloat16)
        s["scale"] = D ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((s["rows"], case["q_heads"]), device="cuda")
    elif op == "turn4":
        _nodes(case, s)
        shape = (layers, s["rows"], H, D)
        s["k_new"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        s["v_new"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        paths = _paths(case)
        s["counts"] = s["node_offsets"].diff()
        s["path"] = torch.tensor([p + [-1] * (s["nmax"] - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        s["accept_len"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        s["new_len"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["ok"] = torch.empty(rows, dtype=torch.int32, device="cuda")
    else:
        s["src"] = torch.tensor(_sources(case), dtype=torch.int32, device="cuda")
        s["ok"] = torch.empty(1, dtype=torch.int32, device="cuda")
    if own:
        import speculative_decoding_verification_74_gb300 as sv
        s["cache"] = (sv.PagedCache4(s["pool"], refs, table, ps, D, k_scale=s["k_scale"], v_scale=s["v_scale"]) if bits == 4
                      else sv.PagedCache(s["k"], s["v"], refs, table))
        if op == "attend4":
            s["ws"] = sv.attention_workspace(s["cache"], case["q_heads"])
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    if s["op"] == "attend4":
        return _plain_attend(s)
    if s["op"] == "beam":
        return _plain_beam(s)
    if s["op"] == "turn4":
        _plain_reserve(s)
        _plain_append(s)
        _plain_commit(s)
    else:
        _plain_reorder(s)
    return _cache_state(s)


def _cache_state(s):
    out = dict(page_refs=s["page_refs"], page_table=s["page_table"], ok=s["ok"],
               length=s["new_len"] if s["op"] == "turn4" else s["seq_len"])
    if "pool" in s:
        out["pool"] = s["pool"]
    else:
        out.update(k=s["k"].view(torch.int16), v=s["v"].view(torch.int16))   # moved as bits
    return out


def _own(s):
    import speculative_decoding_verification_74_gb300 as sv
    if s["op"] == "attend4":
        out, lse = sv.tree_attention(s["q"], s["cache"], 0, s["seq_len"], s["node_offsets"], s["parent"], s["nmax"],
                                     scale=s["scale"], window=s["case"]["window"], sinks=s["case"]["sinks"], out=s["out"],
                                     lse=s["lse"], ws=s["ws"])
        return dict(out=out, lse=lse)
    if s["op"] == "beam":
        scores, rows, tokens = sv.beam_select(s["logits"], s["scores"], s["case"]["candidates"], finished=s["finished"],
                                              pad=s["pad"], ws=s["ws"])
        return dict(scores=scores, rows=rows, tokens=tokens)
    cache = s["cache"]
    if s["op"] == "turn4":
        cache.reserve(s["seq_len"], s["counts"], ok=s["ok"])
        cache.append(s["k_new"], s["v_new"], s["seq_len"], s["node_offsets"])
        cache.commit(s["seq_len"], s["node_offsets"], s["path"], s["accept_len"], out_len=s["new_len"])
    else:
        cache.reorder(s["seq_len"], s["src"], ok=s["ok"])
    return _cache_state(s)


# ---- the 4-bit format --------------------------------------------------------------------

def _regions(pool, D):
    """Views of a pool by group of eight slots: key codes [..., 8, D / 2], key scales [..., 8, D / 16], value codes
    [..., 8 eighths, 4 pairs, 2, D / 16], value scales [..., D / 16, 8]."""
    p = pool.unflatten(-1, (-1, 9 * D))
    a, b, c = 4 * D, 4 * D + D // 2, 8 * D + D // 2
    return (p[..., :a].unflatten(-1, (8, D // 2)), p[..., a:b].unflatten(-1, (8, D // 16)),
            p[..., b:c].unflatten(-1, (8, 4, 2, D // 16)), p[..., c:].unflatten(-1, (D // 16, 8)))


def _quantise(x, whole_scale):
    """Codes [..., D / 2] and scales [..., D / 16] as bytes."""
    inverse = torch.ones((), device="cuda") / torch.full((), whole_scale, device="cuda")
    t = (x.float() * inverse).unflatten(-1, (-1, 16))
    scale = (t.abs().amax(-1) * torch.full((), SIXTH, device="cuda")).clamp(max=448.0).to(torch.float8_e4m3fn)
    by = scale.float().unsqueeze(-1)
    r = torch.where(by > 0, t / by, torch.zeros_like(t))
    a = r.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() +
            (a >= 3.5).byte() + (a > 5.0).byte() + 8 * (torch.signbit(x).unflatten(-1, (-1, 16)) & (by > 0)).byte())
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _values(codes, scales):
    """What codes [..., n bytes] stand for; scales broadcast over [..., 2 n]."""
    steps = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device="cuda")
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return steps[both.int()] * scales


def _write(pool, D, page, slot, k, v):
    """k, v: codes and scales [layers, rows, heads, ...] into each row's slot."""
    kc, ks, vc, vs = _regions(pool, D)
    o, i = slot // 8, slot % 8
    rows_first = lambda t: t.transpose(0, 1)  # noqa: E731
    kc[:, page, :, o, i] = rows_first(k[0])
    ks[:, page, :, o, i] = rows_first(k[1])
    vc[:, page, :, o, :, i // 2, i % 2] = rows_first(v[0].unflatten(-1, (8, -1)))
    vs[:, page, :, o, :, i] = rows_first(v[1])


# ---- attention ---------------------------------------------------------------------------

def _plain_attend(s):
    pool, q = s["pool"][0], s["q"].float()
    ps, lens, table = s["case"]["page_size"], s["seq_len"].long(), s["page_table"].long()
    B, N, Hq, Hk, D = lens.numel(), s["nmax"], q.shape[1], pool.shape[1], q.shape[2]
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
    own_node = (j >= 0) & (j < count[:, None])
    inside = j.clamp(0, N - 1)
    seen = torch.where(cached[:, None, :], True, family.gather(2, inside[:, None, :].expand(B, N, S)) & own_node[:, None, :])
    window, sinks = s["case"]["window"], s["case"]["sinks"]
    if window > 0:
        position = torch.where(cached, slot, lens[:, None] + depth.gather(1, inside))[:, None, :]
        seen &= (position < sinks) | (position > (lens[:, None] + depth)[:, :, None] - window)
    held = pool[table.clamp(min=0)]                                      # [B, entries, Hk, bytes]
    kc, ks, vc, vs = _regions(held, D)
    scale_of = lambda t: t.contiguous().view(torch.float8_e4m3fn).float()  # noqa: E731
    kk = _values(kc, scale_of(ks).repeat_interleave(16, -1))             # [B, entries, Hk, groups, 8, D]
    kk = kk.permute(0, 2, 5, 1, 3, 4).reshape(B, Hk, D, S) * s["k_scale"]
    vv = _values(vc, 1.0).permute(0, 1, 2, 3, 5, 6, 4, 7).flatten(6).flatten(4, 5)
    vv = vv * scale_of(vs).transpose(-1, -2).repeat_interleave(16, -1)
    vv = vv.permute(0, 2, 1, 3, 4, 5).reshape(B, Hk, S, D) * s["v_scale"]
    vv = torch.where((slot < (lens + count)[:, None])[:, None, :, None], vv, 0.0)
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


# ---- beam search -------------------------------------------------------------------------

def _plain_beam(s):
    B, W = s["scores"].shape
    K, V = s["case"]["candidates"], s["logits"].shape[1]
    # 64 bits: candidates of different beams lie next to each other
    x, score = s["logits"].double().view(B, W, V), s["scores"].double()
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    total = torch.where((x > -math.inf) & (score > -math.inf)[:, :, None], score[:, :, None] + (x - lse), -math.inf)
    if s["finished"] is not None:
        done = s["finished"] != 0
        total.masked_fill_(done[:, :, None], -math.inf)
        total[:, :, s["pad"]] = torch.where(done, score, total[:, :, s["pad"]])
    flat = total.view(B, W * V)
    least = flat.topk(min(K, W * V)).values[:, -1:]
    b, at = torch.nonzero((flat >= least) & (flat > -math.inf), as_tuple=True)
    order = torch.sort(flat[b, at], descending=True, stable=True).indices  # then by request: ties keep their order
    order = order[torch.sort(b[order], stable=True).indices]
    b, at = b[order], at[order]
    count = torch.bincount(b, minlength=B)
    place = torch.arange(b.numel(), device="cuda") - (count.cumsum(0) - count)[b]
    b, at, place = b[place < K], at[place < K], place[place < K]
    out = dict(scores=torch.full((B, K), -math.inf, device="cuda"),
               rows=torch.full((B, K), -1, dtype=torch.int32, device="cuda"),
               tokens=torch.full((B, K), -1, dtype=torch.int32, device="cuda"))
    out["scores"][b, place] = flat[b, at].float()
    out["rows"][b, place] = (b * W + at // V).int()
    out["tokens"][b, place] = (at % V).int()
    return out


# ---- the cache ---------------------------------------------------------------------------

def _need(s, length):
    return (length.long() + s["case"]["page_size"] - 1) // s["case"]["page_size"]


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
    ps = s["case"]["page_size"]
    return s["page_table"].long()[request, slot // ps], slot % ps


def _plain_append(s):
    B = s["seq_len"].numel()
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), s["counts"].long(), output_size=s["rows"])
    c = torch.arange(s["rows"], device="cuda") - s["node_offsets"].long()[b]
    page, slot = _places(s, b, s["seq_len"].long()[b] + c)
    _write(s["pool"], s["case"]["head_dim"], page, slot, _quantise(s["k_new"], s["k_scale"]), _quantise(s["v_new"], s["v_scale"]))


def _plain_commit(s):
    lens, path = s["seq_len"].long(), s["path"].long()
    b, j = torch.nonzero(torch.arange(path.shape[1], device="cuda") < s["accept_len"][:, None], as_tuple=True)
    page, slot = _places(s, b, lens[b] + path[b, j])
    kc, ks, vc, vs = _regions(s["pool"], s["case"]["head_dim"])
    o, i = slot // 8, slot % 8
    layers_first = lambda t: t.transpose(0, 1)  # noqa: E731
    k = layers_first(kc[:, page, :, o, i]), layers_first(ks[:, page, :, o, i])
    v = layers_first(vc[:, page, :, o, :, i // 2, i % 2].flatten(-2)), layers_first(vs[:, page, :, o, :, i])
    to_page, to_slot = _places(s, b, lens[b] + 1 + j)
    _write(s["pool"], s["case"]["head_dim"], to_page, to_slot, k, v)
    s["new_len"].copy_(lens + torch.where(s["accept_len"] >= 0, s["accept_len"] + 1, 0))
    table = s["page_table"]
    back = (torch.arange(table.shape[1], device="cuda") >= _need(s, s["new_len"])[:, None]) & (table >= 0)
    s["page_refs"].index_add_(0, table[back].long(), torch.full_like(table[back], -1))
    table.masked_fill_(back, -1)


def _plain_reorder(s):
    """Beam j goes on from src[j]: full pages are shared; of the beams that go on from one sequence, itself or else the
    first keeps its partly filled page, and the others get copies in the lowest free pages, in order."""
    src, table, refs, lens = s["src"].long(), s["page_table"], s["page_refs"], s["seq_len"].long()
    R, ps = table.shape[0], s["case"]["page_size"]
    row = torch.arange(R, device="cuda")
    first = torch.full((R,), R, device="cuda").scatter_reduce(0, src, row, "amin")
    keeper = torch.where(src == row, row, torch.where(src[src] == src, src, first[src]))
    keeps = keeper == row
    new_len, old = lens[src], table.long()[src]
    full, part = new_len // ps, new_len % ps
    entry = torch.arange(table.shape[1], device="cuda")
    rows = torch.where(keeps[:, None] | (entry < full[:, None]), old, -1)
    held = table[table >= 0].long()
    counts = refs.clone().index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    kept = rows[rows >= 0]
    counts.index_add_(0, kept, torch.ones_like(kept, dtype=torch.int32))
    copies = torch.nonzero(~keeps & (part > 0)).flatten()
    page = torch.nonzero(counts == 0).flatten()[:copies.numel()]
    source = old[copies, full[copies]]
    rows[copies, full[copies]] = page
    counts[page] = 1
    if "pool" in s:                                                      # whole groups of eight slots
        used = torch.arange(ps // 8, device="cuda") < ((part[copies] + 7) // 8)[:, None]
        held = s["pool"].unflatten(-1, (ps // 8, -1))
        held[:, page] = torch.where(used[None, :, None, :, None], held[:, source], held[:, page])
    else:
        used = (torch.arange(ps, device="cuda") < part[copies][:, None])[None, :, :, None, None]
        s["k"][:, page] = torch.where(used, s["k"][:, source], s["k"][:, page])
        s["v"][:, page] = torch.where(used, s["v"][:, source], s["v"][:, page])
    table.copy_(rows)
    refs.copy_(counts)
    s["seq_len"].copy_(new_len)
    s["ok"].fill_(1)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "beam":
        rows = case["requests"] * case["beams"]
        n = rows * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 8 * rows + 12 * case["requests"] * case["candidates"],
                "flops": 4 * n}
    four = case["kv_heads"] * case["head_dim"] * 9 // 8                  # a token's keys and values in one layer, 4 bits
    wide = case["kv_heads"] * case["head_dim"] * 2 * 2                   # the same in bf16
    if case["op"] == "attend4":
        slots = pairs = rows = 0
        for n, parent in zip(_lengths(case, case["requests"]), _parents(case)):
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
        return {"bytes": slots * four + rows * (2 * row + 4 * case["q_heads"]),
                "flops": 4 * case["q_heads"] * case["head_dim"] * pairs}
    if case["op"] == "turn4":
        rows = sum(len(p) for p in _parents(case))
        moved = sum(1 for path in _paths(case) for j, node in enumerate(path) if node != j + 1)
        return {"bytes": case["layers"] * (rows * (wide + four) + 2 * moved * four), "flops": 0}
    src, rows = _sources(case), case["requests"] * case["beams"]
    lens = _lengths(case, rows)
    kept = {}                                                            # one beam of each source moves nothing
    for j, p in enumerate(src):
        kept.setdefault(p, j)
    slots = sum(lens[p] % case["page_size"] for j, p in enumerate(src) if kept[p] != j)
    entries = sum(-(-n // case["page_size"]) for n in lens)
    return {"bytes": 2 * slots * case["layers"] * (four if case["bits"] == 4 else wide) + 8 * entries + 12 * rows, "flops": 0}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] not in ("attend4", "beam"):
        return None                                                      # bytes and whole numbers
    s = prepare(case, seed)
    return _exact_attend(s) if case["op"] == "attend4" else _exact_beam(s)


def _decoded(s, page, slot):
    """Keys and values [slots, heads, D] of the given slots, byte by byte as the format says."""
    D, pool = s["case"]["head_dim"], s["pool"][0]
    d = torch.arange(D, device="cuda")
    base, i, eighth = (slot // 8 * 9 * D)[:, None], (slot % 8)[:, None], D // 8
    read = lambda at: pool[page].gather(2, at[:, None, :].expand(-1, pool.shape[1], -1)).long()  # noqa: E731

    def number(byte_at, scale_at):
        code = (read(byte_at) >> (4 * (d % 2))) & 15
        e, m = (code >> 1) & 3, (code & 1).double()
        value = torch.where(e > 0, (1 + m / 2) * 2.0 ** (e - 1).double(), m / 2) * torch.where(code >= 8, -1.0, 1.0).double()
        b = read(scale_at)
        e, m = b >> 3, (b & 7).double()                                  # e4m3 without a sign
        return value * torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7).double(), m / 8 * 2.0 ** -6)

    k = number(base + i * (D // 2) + d // 2, base + 4 * D + i * (D // 16) + d // 16)
    v = number(base + 4 * D + D // 2 + (d // eighth * 4 + i // 2) * eighth + i % 2 * (eighth // 2) + d % eighth // 2,
               base + 8 * D + D // 2 + d // 16 * 8 + i)
    return k * s["k_scale"], v * s["v_scale"]


def _exact_attend(s):
    """Request by request, head group by head group, over the slots that a node's path can see."""
    case = s["case"]
    ps, G = case["page_size"], case["q_heads"] // case["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty((s["rows"], case["q_heads"]), dtype=torch.float64, device="cuda")
    lens, table = s["seq_len"].tolist(), s["page_table"].long()
    first = 0
    for i, parent in enumerate(_parents(case)):
        L, N = lens[i], len(parent)
        slots = torch.arange(L + N, device="cuda")
        halves = [_decoded(s, table[i, part // ps], part % ps) for part in slots.split(8192)]
        keys, values = torch.cat([h[0] for h in halves]), torch.cat([h[1] for h in halves])  # [S, Hk, D]
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


def _exact_beam(s):
    """Request by request: the largest sums of a beam's score and its row's log-softmax."""
    B, W = s["scores"].shape
    K = s["case"]["candidates"]
    scores = torch.full((B, K), -math.inf, dtype=torch.float64, device="cuda")
    for i in range(B):
        candidates = []
        for w in range(W):
            if s["finished"] is not None and s["finished"][i, w]:
                candidates.append(s["scores"][i, w:w + 1].double())
            else:
                row = torch.log_softmax(s["logits"][i * W + w].double(), 0) + s["scores"][i, w].double()
                candidates.append(torch.sort(row, descending=True).values[:K])
        best = torch.sort(torch.cat(candidates), descending=True).values[:K]
        scores[i, :best.numel()] = best
    return dict(scores=scores, rows=None, tokens=None)
