"""Sampling with temperature, top-k, top-p and min-p, in float64 with real-valued weights.

Row by row: softmax(x / T); tokens in the order (logit desc, index asc); top-k keeps the first k;
top-p those whose mass before them is below p of the top-k's mass; min-p those of at least q times
the largest weight; draws by inverse CDF in vocabulary order over what is kept.
"""
from __future__ import annotations

import numpy as np


def sample_row(x, T, k, p, q, uniforms, band=2e-6):
    """One row (float64 logits, -inf = masked).  Returns a dict:
    tokens [M] (-1 for an empty row), probs [M], kept [V] bool,
    near_draw [M]: the draw lies within band of a bin edge,
    near_cut: token indices whose membership hangs on a difference below band (in mass or weight)."""
    x = np.asarray(x, np.float64)
    V, M = len(x), len(uniforms)
    if not np.any(x > -np.inf):
        return dict(tokens=np.full(M, -1), probs=np.zeros(M), kept=np.zeros(V, bool), near_draw=np.zeros(M, bool),
                    near_cut=np.zeros(0, int))
    order = np.lexsort((np.arange(V), -x))
    near = []
    if T == 0:
        keep_sorted = np.arange(V) < 1
        e = np.zeros(V)
        e[order[0]] = 1.0
    else:
        e = np.exp((x - x.max()) / T)
        es = e[order]
        keep_sorted = np.ones(V, bool)
        if k > 0:
            keep_sorted[k:] = False
        W = (es * keep_sorted).sum()
        if p < 1:
            before = np.cumsum(es * keep_sorted) - es * keep_sorted
            near += list(order[(np.abs(before - p * W) < band * W) & keep_sorted])
            keep_sorted &= before < p * W
            keep_sorted[0] = True
        if q > 0:
            near += list(order[np.abs(np.log2(np.maximum(es, 1e-300)) - np.log2(q)) < 1e-5])
            keep_sorted &= es >= q
    kept = np.zeros(V, bool)
    kept[order] = keep_sorted
    kept &= x > -np.inf
    w = e * kept
    c = np.cumsum(w)
    Z = c[-1]
    tokens, probs, near_draw = np.empty(M, int), np.empty(M), np.zeros(M, bool)
    for j, u in enumerate(uniforms):
        t = u * Z
        y = int(np.searchsorted(c, t, side="right"))
        y = min(y, int(np.nonzero(w > 0)[0][-1]))
        tokens[j], probs[j] = y, w[y] / Z
        near_draw[j] = abs(c[y] - t) < band * Z or abs((c[y - 1] if y else 0.0) - t) < band * Z and y > 0
    return dict(tokens=tokens, probs=probs, kept=kept, near_draw=near_draw, near_cut=np.asarray(near, int))
