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


def linear_xent(x, w, targets, smoothing=0.0, z=0.0, ignore=-100):
    """(loss, lse) of each row; 0 for rows to be ignored, NaN for targets outside the vocabulary."""
    logits = x @ w.T
    with np.errstate(all="ignore"):
        top = logits.max(1)
        lse = top + np.log(np.exp(logits - top[:, None]).sum(1))
    loss = np.empty(len(x))
    for i, t in enumerate(targets):
        if t == ignore:
            loss[i] = lse[i] = 0.0
        elif not 0 <= t < len(w):
            loss[i] = lse[i] = np.nan
        else:
            loss[i] = lse[i] - (1 - smoothing) * logits[i, t] - smoothing * logits[i].mean() + z * lse[i] ** 2
    return loss, lse


def xent_slope(dloss, x, w, targets, lse, smoothing=0.0, z=0.0, ignore=-100):
    """Gradient with respect to the logits, and exp(logits - lse)."""
    rows = [i for i, t in enumerate(targets) if t != ignore and 0 <= t < len(w)]
    d, p = np.zeros((len(x), len(w))), np.zeros((len(x), len(w)))
    for i in rows:
        p[i] = np.exp(w @ x[i] - lse[i])
        d[i] = p[i] * (1 + 2 * z * lse[i]) - smoothing / len(w)
        d[i, targets[i]] -= 1 - smoothing
        d[i] *= dloss[i]
    return d, p


def linear_xent_bwd(dloss, x, w, targets, lse, smoothing=0.0, z=0.0, ignore=-100):
    """(dx, dw)."""
    d, _ = xent_slope(dloss, x, w, targets, lse, smoothing, z, ignore)
    rows = [i for i in range(len(x)) if d[i].any()]
    return d @ w, d[rows].T @ x[rows]
