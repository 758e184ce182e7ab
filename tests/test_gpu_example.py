"""The example that runs sampling, the paged cache, tree attention and tree verification together."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu

PROMPT_LENGTHS = [1, 7, 16, 33]


@pytest.fixture(scope="module")
def example():
    import tree_round
    return tree_round


def prompts(model):
    g = torch.Generator().manual_seed(3)
    return [torch.randint(model.vocab, (n,), generator=g).tolist() for n in PROMPT_LENGTHS]


def dense_logits(example, model, text):
    """The model over a whole text with plain attention in float32."""
    n, group = len(text), model.q_heads // model.kv_heads
    hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)

    def attend(_, q, k, v):
        k, v = (t.float().repeat_interleave(group, 1) for t in (k, v))
        x = torch.einsum("qhd,khd->hqk", q.float(), k) * model.head_dim ** -0.5
        return torch.einsum("hqk,khd->qhd", x.masked_fill(hidden, float("-inf")).softmax(-1), v).to(q.dtype)

    return model.forward(torch.tensor(text, device="cuda"), torch.arange(n, device="cuda"), attend).float()


@pytest.mark.parametrize("branching", [(1,), (2, 2, 1), (5, 1)])
def test_greedy_text_is_the_targets_own(example, branching):
    # every token is a largest logit of the dense model up to bf16's rounding: activations and logits carry 8 bits, so
    # two computations differ by a few parts in 2^8 of a logit's spread; 2^-4 of it bounds that
    model = example.Model()
    start = prompts(model)
    texts, rounds = example.generate(model, start, 24, 0.0, branching=branching)
    for p, text in zip(start, texts):
        logits = dense_logits(example, model, text)[len(p) - 1:-1]
        took = logits.gather(1, torch.tensor(text[len(p):], device="cuda")[:, None]).squeeze(1)
        assert len(text) - len(p) >= 24
        assert bool((took >= logits.amax(1) - logits.std(1) * 2.0 ** -4).all())


def test_sampled_texts_are_repeatable_and_differ_by_seed(example):
    model = example.Model()
    start = prompts(model)
    run = lambda seed: example.generate(model, start, 16, 0.9, top_k=40, top_p=0.9, seed=seed)  # noqa: E731
    a, b, c = run(0), run(0), run(1)
    assert a == b and a != c
    assert all(0 <= t < model.vocab for text in a[0] for t in text)
