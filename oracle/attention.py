"""Attention of a token tree over a paged cache, in float64, one query row and head at a time."""
from __future__ import annotations

import numpy as np


def path_of(parent, c):
    """Node c's ancestors and itself, root first (parent None = a chain)."""
    line = [c]
    while line[-1] > 0:
        line.append(line[-1] - 1 if parent is None else int(parent[line[-1]]))
    return line[::-1]


def tree_attention(q, k, v, page_table, seq_len, node_offsets, parent, scale, window=0, sinks=0):
    """q [rows, Hq, D]; k, v [pages, page_size, Hk, D] (float64); returns (out [rows, Hq, D], lse [rows, Hq])."""
    rows, Hq, D = q.shape
    ps, Hk = k.shape[1], k.shape[2]
    out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    for i in range(len(seq_len)):
        a, b, L = int(node_offsets[i]), int(node_offsets[i + 1]), int(seq_len[i])
        tree = None if parent is None else parent[a:b]
        for c in range(b - a):
            path = path_of(tree, c)
            here = L + len(path) - 1
            slots, positions = list(range(L)) + [L + n for n in path], list(range(here + 1))
            if window > 0:
                slots = [s for s, p in zip(slots, positions) if p < sinks or p > here - window]
            slots = np.asarray(slots)
            pages = page_table[i, slots // ps]
            for h in range(Hq):
                g = h // (Hq // Hk)
                x = scale * (k[pages, slots % ps, g] @ q[a + c, h])
                m = x.max()
                e = np.exp(x - m)
                out[a + c, h] = e @ v[pages, slots % ps, g] / e.sum()
                lse[a + c, h] = m + np.log(e.sum())
    return out, lse
