"""Speculative decoding with token trees over a paged cache, end to end on a small random model: per round

    drafter   sample()  candidates of each node, level by level, and the rows they were drawn from
    target    PagedCache.reserve / append and tree_attention() over all nodes of all requests
              sample()  the target's rows cut by the same filters
    verify_tree()       the accepted path of every request
    PagedCache.commit   keeps that path's keys and values, gives the pages past it back

The drafter is the target's first layer.  With temperature 0 the text is the target's own greedy text.

    python examples/tree_round.py [--requests 8] [--new-tokens 64] [--temperature 0.8] [--cache-bits 4]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_74_gb300 as sv  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32
BRANCHING = (2, 2, 1)  # children of every node, level by level


class Model:
    """A few layers of grouped-query attention and gated feed-forward with rotary positions and random weights."""

    def __init__(self, vocab=1000, width=256, layers=2, q_heads=4, kv_heads=2, head_dim=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: (torch.randn(s, generator=g, device="cuda") / s[-1] ** 0.5).to(BF16)  # noqa: E731
        self.vocab, self.q_heads, self.kv_heads, self.head_dim = vocab, q_heads, kv_heads, head_dim
        self.embed, self.head = w(vocab, width) * width ** 0.5, w(vocab, width) * 3
        self.layers = [dict(q=w(q_heads * head_dim, width), k=w(kv_heads * head_dim, width), v=w(kv_heads * head_dim, width),
                            o=w(width, q_heads * head_dim), up=w(2 * width, width), down=w(width, width) * (1.0 if i == 0 else 0.25))
                       for i in range(layers)]

    def first_layer(self):
        m = object.__new__(Model)
        m.__dict__.update(self.__dict__, layers=self.layers[:1])
        return m

    def cache(self, requests, longest, page_size=16, bits=16):
        entries = -(-longest // page_size)
        kind = sv.PagedCache4 if bits == 4 else sv.PagedCache
        return kind.empty(len(self.layers), requests * entries, page_size, self.kv_heads, self.head_dim, requests, entries)

    def _rotate(self, x, position):
        half = self.head_dim // 2
        angle = position[:, None, None] * 10000.0 ** (-torch.arange(half, device=x.device) / half)
        a, b = x.float().split(half, -1)
        return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1).to(BF16)

    def forward(self, tokens, position, attend):
        """Logits [rows, vocab]; attend(layer, q, k, v) is the attention, [rows, heads, head_dim]."""
        x = self.embed[tokens.long()]
        norm = lambda x: F.rms_norm(x.float(), x.shape[-1:]).to(BF16)  # noqa: E731
        for i, w in enumerate(self.layers):
            h = norm(x)
            q, k, v = ((h @ w[n].T).view(len(h), -1, self.head_dim) for n in "qkv")
            x = x + attend(i, self._rotate(q, position), self._rotate(k, position), v).flatten(1) @ w["o"].T
            gate, up = (norm(x) @ w["up"].T).chunk(2, -1)
            x = x + (F.silu(gate) * up) @ w["down"].T
        return norm(x) @ self.head.T


class Side:
    """A model with its cache and workspaces: the drafter's or the target's side of a round."""

    def __init__(self, model, requests, longest, bits=16):
        self.model, self.cache = model, model.cache(requests, longest, bits=bits)
        self.ws = sv.attention_workspace(self.cache, model.q_heads)

    def run(self, tokens, depth, seq_len, offsets, parent, nmax):
        """Logits of all nodes: their keys and values go into the cache, each node sees its request's sequence and its
        own path."""
        request = torch.repeat_interleave(torch.arange(len(seq_len), device="cuda"), offsets.diff())

        def attend(layer, q, k, v):
            self.cache.append(k, v, seq_len, offsets, layer)
            return sv.tree_attention(q, self.cache, layer, seq_len, offsets, parent, nmax, lse=False, ws=self.ws)[0]

        return self.model.forward(tokens, seq_len[request] + depth, attend)


def tree_of(branching):
    """(parents, depths, first node of each level) of a full tree, level by level."""
    parent, depth, levels = [-1], [0], [0]
    for level, children in enumerate(branching):
        first = levels[-1]
        levels.append(len(parent))
        for node in range(first, levels[-1]):
            parent += [node] * children
            depth += [level + 1] * children
    return parent, depth, levels


def generate(model, prompts, new_tokens, temperature, *, top_k=0, top_p=1.0, branching=BRANCHING, seed=0, bits=16):
    """Continues the prompts (lists of token ids) by at least new_tokens tokens each, with caches held in 16 or 4
    bits.  Returns (texts, rounds)."""
    B = len(prompts)
    parents, depths, levels = tree_of(branching)
    N = len(parents)
    longest = max(map(len, prompts)) + new_tokens + 2 * N
    target, drafter = Side(model, B, longest, bits), Side(model.first_layer(), B, longest, bits)
    gpu = lambda x, dtype=I32: torch.tensor(x, dtype=dtype, device="cuda")  # noqa: E731
    # the prompts but their last tokens: chains over empty sequences
    seq_len, counts = gpu([0] * B), [len(p) - 1 for p in prompts]
    offsets = gpu([0] + counts).cumsum(0, dtype=I32)
    if sum(counts):
        for side in (drafter, target):
            side.cache.reserve(seq_len, gpu(counts))
            side.run(gpu([t for p in prompts for t in p[:-1]]), gpu([c for n in counts for c in range(n)]), seq_len, offsets, None,
                     max(counts))
    seq_len, root = gpu(counts), gpu([p[-1] for p in prompts])

    T = torch.full((B,), float(temperature), device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    filters = lambda rows: dict(top_k=torch.full((rows,), top_k, dtype=I32, device="cuda"),  # noqa: E731
                                top_p=torch.full((rows,), top_p, device="cuda"))
    whole = torch.arange(B + 1, dtype=I32, device="cuda") * N
    parent, depth, more = gpu(parents * B), gpu(depths * B), gpu([N] * B)
    texts, rounds = [list(p) for p in prompts], 0
    while min(len(t) - len(p) for t, p in zip(texts, prompts)) < new_tokens:
        for side in (drafter, target):
            side.cache.reserve(seq_len, more)
        tokens = torch.zeros(B, N, dtype=I32, device="cuda")
        tokens[:, 0] = root
        draft_rows = torch.zeros(B, N, model.vocab, dtype=BF16, device="cuda")
        for level, first in enumerate(levels):
            n = levels[level + 1] if level + 1 < len(levels) else N  # nodes so far (again with each level: they are few)
            here = torch.arange(B + 1, dtype=I32, device="cuda") * n
            logits = drafter.run(tokens[:, :n].flatten(), gpu(depths[:n] * B), seq_len, here, gpu(parents[:n] * B), n)
            if n == N:
                break
            # candidates are drawn, never repeated greedily: at temperature 0 verification only compares them
            rows = logits.view(B, n, -1)[:, first:].flatten(0, 1)
            children = branching[level]
            u = torch.rand(len(rows), children, generator=gen, device="cuda").clamp(max=1 - 2.0 ** -24)
            drawn, _, cut = sv.sample(rows, torch.full((len(rows),), float(temperature) or 1.0, device="cuda"), u, probs=False,
                                      filtered=True, **filters(len(rows)))
            tokens[:, n:n + (n - first) * children] = drawn.view(B, -1)
            draft_rows[:, first:n] = cut.view(B, n - first, -1)
        logits = target.run(tokens.flatten(), depth, seq_len, whole, parent, N)
        rows = sv.sample(logits, T.repeat_interleave(N), torch.empty(B * N, 0, device="cuda"), probs=False, filtered=True,
                         **filters(B * N))[2]
        path, out, accepted, _ = sv.verify_tree(rows, draft_rows.flatten(0, 1), whole, parent, tokens.flatten(), T, N, seed=seed,
                                                round_=rounds)
        drafter.cache.commit(seq_len, whole, path, accepted)
        seq_len = target.cache.commit(seq_len, whole, path, accepted)
        root = out.gather(1, accepted.long()[:, None]).squeeze(1)
        for text, row, a in zip(texts, out.tolist(), accepted.tolist()):
            text += row[:a + 1]
        rounds += 1
    for side in (drafter, target):
        for ws in (side.cache.ws, side.ws):
            status, word = sv.sv_query_status(ws)
            if status != sv.SV_OK:
                raise RuntimeError(f"device status {word:#x}")
    return texts, rounds


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--requests", type=int, default=8)
    a.add_argument("--new-tokens", type=int, default=64)
    a.add_argument("--temperature", type=float, default=0.8)
    a.add_argument("--cache-bits", type=int, choices=(16, 4), default=16)
    a = a.parse_args()
    model = Model()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(model.vocab, (int(n),), generator=g).tolist() for n in torch.randint(1, 40, (a.requests,), generator=g)]
    generate(model, prompts, 4, a.temperature, bits=a.cache_bits)  # warm-up
    torch.cuda.synchronize()
    began = time.time()
    texts, rounds = generate(model, prompts, a.new_tokens, a.temperature, top_k=50, top_p=0.95, bits=a.cache_bits)
    new = sum(len(t) - len(p) for t, p in zip(texts, prompts))
    print(f"{a.requests} requests, {new} tokens in {rounds} rounds: {new / rounds / a.requests:.2f} tokens a request and round, "
          f"{(time.time() - began) / rounds * 1e3:.2f} ms a round")
    print("first text:", texts[0][len(prompts[0]):][:16])


if __name__ == "__main__":
    main()
