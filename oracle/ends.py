"""fp64 oracles of the two ends of a training step (numpy; written from the definitions): the embedding and its gradient, the
softmax cross entropy of the output projection and its gradients.

Inputs are float64 arrays that hold the bf16 / fp16 / fp32 values exactly.
"""
from __future__ import annotations

import numpy as np


def embedding(ids, w, scale=1.0):
    """Rows of w [V, K]; NaN for an id outside the table."""
    out = np.full((len(ids), w.shape[1]), np.nan)
    for i, v in enumerate(ids):
        if 0 <= v < len(w):
            out[i] = scale * w[v]
    return out


def embedding_bwd(dy, ids, n_rows, scale=1.0, padding=None, dw=None):
    """The table's gradient, added to dw if that is given; and the number of rows and the sum of sizes behind each element."""
    out = np.zeros((n_rows, dy.shape[1]))
    count, size = np.zeros(n_rows, dtype=np.int64), np.zeros_like(out)
    for i, v in enumerate(ids):
        if 0 <= v < n_rows and v != padding:
            out[v] += scale * dy[i]
            size[v] += np.abs(scale * dy[i])
            count[v] += 1
    if dw is not None:
        out, size = out + dw, size + np.abs(dw)
    return out, count, size
