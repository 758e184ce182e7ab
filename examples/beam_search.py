"""Beam search over a paged cache held in 16 or 4 bits, end to end on a small random model: per step

    PagedCache.reserve / append and tree_attention()    the beams' last tokens, one node each
    beam_select()                                       the best continuations over beams and vocabulary
    PagedCache.reorder                                  every sequence becomes a copy of the one that its beam goes on from

    python examples/beam_search.py [--requests 8] [--beams 4] [--new-tokens 64] [--cache-bits 4]
"""
from __future__ import annotations

import argparse
import time

import torch
from tree_round import I32, Model, sv


def search(model, prompts, beams, new_tokens, *, bits=16, end=None):
    """The `beams` best continuations of each prompt (lists of token ids), new_tokens tokens long or, where a beam takes the
    token `end`, shorter.  Returns (texts [requests][beams], scores [requests, beams]), best first."""
    B, W = len(prompts), beams
    gpu = lambda x, dtype=I32: torch.tensor(x, dtype=dtype, device="cuda")  # noqa: E731
    longest = max(map(len, prompts)) + new_tokens
    cache = model.cache(B * W, longest, bits=bits)
    ws = sv.attention_workspace(cache, model.q_heads)

    def logits_of(tokens, position, seq_len, offsets, nmax):
        def attend(layer, q, k, v):
            cache.append(k, v, seq_len, offsets, layer)
            return sv.tree_attention(q, cache, layer, seq_len, offsets, None, nmax, lse=False, ws=ws)[0]

        return model.forward(tokens, position, attend)

    # the prompts but their last tokens, each in the row of its request's first beam, then in all of them
    counts = [len(p) - 1 if w == 0 else 0 for p in prompts for w in range(W)]
    offsets, seq_len = gpu([0] + counts).cumsum(0, dtype=I32), gpu([0] * (B * W))
    if sum(counts):
        cache.reserve(seq_len, gpu(counts))
        logits_of(gpu([t for p in prompts for t in p[:-1]]), gpu([c for n in counts for c in range(n)]), seq_len, offsets, max(counts))
    seq_len = gpu(counts)
    cache.reorder(seq_len, torch.arange(B * W, dtype=I32, device="cuda") // W * W)

    scores = torch.full((B, W), -torch.inf, device="cuda")
    scores[:, 0] = 0                                        # one beam at first
    tokens, one = gpu([p[-1] for p in prompts]).repeat_interleave(W), gpu([1] * (B * W))
    offsets = torch.arange(B * W + 1, dtype=I32, device="cuda")
    new = torch.empty((B * W, 0), dtype=I32, device="cuda")
    done = torch.zeros((B, W), dtype=I32, device="cuda")
    beam_ws = sv.beam_workspace(B * W, model.vocab, W)
    for _ in range(new_tokens):
        cache.reserve(seq_len, one)
        logits = logits_of(tokens, seq_len, seq_len, offsets, 1)
        seq_len += 1
        scores, rows, picked = sv.beam_select(logits, scores, W, finished=done, pad=0 if end is None else end, ws=beam_ws)
        cache.reorder(seq_len, rows.flatten())
        came_from = rows.flatten().long().clamp(min=0)      # (-1: fewer candidates than beams)
        tokens = picked.flatten().clamp(min=0)
        new = torch.cat([new[came_from], tokens[:, None]], 1)
        if end is not None:
            done = (done.flatten()[came_from] | (tokens == end)).view(B, W).int()
    for w in (cache.ws, ws, beam_ws):
        status, word = sv.sv_query_status(w)
        if status != sv.SV_OK:
            raise RuntimeError(f"device status {word:#x}")
    texts = [[row[:row.index(end) + 1] if end in row else row for row in request] for request in new.view(B, W, -1).tolist()]
    return texts, scores


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--requests", type=int, default=8)
    a.add_argument("--beams", type=int, default=4)
    a.add_argument("--new-tokens", type=int, default=64)
    a.add_argument("--cache-bits", type=int, choices=(16, 4), default=16)
    a = a.parse_args()
    model = Model()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(model.vocab, (int(n),), generator=g).tolist() for n in torch.randint(1, 40, (a.requests,), generator=g)]
    search(model, prompts, a.beams, 2, bits=a.cache_bits)  # warm-up
    torch.cuda.synchronize()
    began = time.time()
    texts, scores = search(model, prompts, a.beams, a.new_tokens, bits=a.cache_bits)
    print(f"{a.requests} requests, {a.beams} beams, {a.new_tokens} tokens: {(time.time() - began) / a.new_tokens * 1e3:.2f} ms a step")
    print("first text:", texts[0][0][:16], f"log-probability {scores[0, 0].item():.2f}")


if __name__ == "__main__":
    main()
