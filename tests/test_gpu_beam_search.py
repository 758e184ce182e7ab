"""The example that runs append, tree attention, beam selection and reordering together, over both kinds of cache: against a
search whose beams keep private pages and have every page copied, in plain tensor code, when they move.  The attention sees
the same values in the same order whatever page they lie in, so the two searches agree to the bit."""
import os
import sys

import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from oracle.beam import beam_select

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu
PROMPTS = [[5], [7, 1, 2, 3, 4, 5, 6], list(range(16)), list(range(100, 133))]


@pytest.fixture(scope="module")
def examples():
    import beam_search
    import tree_round
    return beam_search, tree_round


def by_private_pages(model, prompts, W, new_tokens, bits, end):
    B = len(prompts)
    entries = -(-(max(map(len, prompts)) + new_tokens) // 16)
    cache = model.cache(B * W, entries * 16, bits=bits)
    cache.page_table.copy_(torch.arange(B * W * entries, dtype=torch.int32, device="cuda").view(B * W, entries))
    cache.page_refs.fill_(1)
    pools = [cache.pool] if bits == 4 else [cache.k, cache.v]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(tokens, position, lens, offsets, nmax):
        def attend(layer, q, k, v):
            cache.append(k, v, lens, offsets, layer)
            return sv.tree_attention(q, cache, layer, lens, offsets, None, nmax)[0]

        return model.forward(i32(tokens), i32(position), attend)

    def move(rows):
        for pool in pools:
            by_row = pool.view(pool.shape[0], B * W, entries, -1)
            by_row.copy_(by_row[:, torch.tensor(rows, device="cuda")].clone())

    counts = [len(p) - 1 if w == 0 else 0 for p in prompts for w in range(W)]
    step([t for p in prompts for t in p[:-1]], [c for n in counts for c in range(n)], i32([0] * (B * W)),
         i32(np.concatenate([[0], np.cumsum(counts)])), max(counts))
    move([i // W * W for i in range(B * W)])
    lens = np.repeat([len(p) - 1 for p in prompts], W)
    scores = np.full((B, W), -np.inf)
    scores[:, 0] = 0
    texts, done = [[] for _ in range(B * W)], np.zeros((B, W), int)
    tokens = [p[-1] for p in prompts for _ in range(W)]
    for _ in range(new_tokens):
        logits = step(tokens, lens, i32(lens), i32(range(B * W + 1)), 1)
        lens = lens + 1
        picked, rows, new = beam_select(logits.double().cpu().numpy(), scores, W, done if end is not None else None, end or 0)
        scores = picked.astype(np.float32).astype(np.float64)
        move(list(rows.flatten()))
        tokens = [int(t) for t in new.flatten()]
        texts = [texts[r] + [t] for r, t in zip(rows.flatten(), tokens)]
        done = np.array([[int(done.flatten()[r] or (end is not None and t == end)) for r, t in zip(*pair)] for pair in zip(rows, new)])
    cut = [t[:t.index(end) + 1] if end in t else t for t in texts]
    return [cut[i * W:(i + 1) * W] for i in range(B)], scores


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("W,end", [(1, None), (4, None), (3, 17)])
def test_search(examples, bits, W, end):
    model = examples[1].Model(vocab=300)
    if end is not None:
        model.head[end] *= 0
        model.head[end] += model.head[40:60].mean(0) * 4     # a token that is taken now and then
    texts, scores = examples[0].search(model, PROMPTS, W, 20, bits=bits, end=end)
    want, want_scores = by_private_pages(model, PROMPTS, W, 20, bits, end)
    assert texts == want
    # each step adds a rounding of its sum to float32 (2^-24 of at most the last score) and the row sums' 2^-18
    assert np.abs(scores.double().cpu().numpy() - want_scores).max() <= 20 * (2.0 ** -24 * np.abs(want_scores).max() + 2.0 ** -18)


def test_rounds_over_a_cache_of_4_bits(examples):
    model = examples[1].Model()
    texts, rounds = examples[1].generate(model, PROMPTS, 16, 0.9, top_k=40, bits=4)
    again, _ = examples[1].generate(model, PROMPTS, 16, 0.9, top_k=40, bits=4)
    assert texts == again and all(len(t) - len(p) >= 16 and t[:len(p)] == p for t, p in zip(texts, PROMPTS))
    assert all(0 <= t < model.vocab for text in texts for t in text)
