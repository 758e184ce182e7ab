"""One step of beam search in float64: every candidate listed, one sort."""
from __future__ import annotations

import numpy as np


def beam_select(logits, scores, candidates, finished=None, pad=0):
    """logits [B * W, V], scores [B, W] (float64); returns (scores, rows, tokens), each [B, candidates]."""
    B, W = scores.shape
    out = np.full((B, candidates), -np.inf), np.full((B, candidates), -1), np.full((B, candidates), -1)
    for i in range(B):
        found = []
        for w in range(W):
            score, row = scores[i, w], logits[i * W + w]
            if score == -np.inf:
                continue
            if finished is not None and finished[i, w]:
                found.append((-score, w, pad))
                continue
            m = row.max()
            if m == -np.inf:
                continue
            total = (row - m) + (score - np.log(np.exp(row - m).sum()))   # (m + log would lose the log beside a large m)
            found += [(-total[v], w, v) for v in np.flatnonzero(row > -np.inf)]
        for j, (t, w, v) in enumerate(sorted(found)[:candidates]):
            out[0][i, j], out[1][i, j], out[2][i, j] = -t, i * W + w, v
    return out
