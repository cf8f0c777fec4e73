"""Oracle of the whole expert layer for a few tokens: CPU, float64."""
from __future__ import annotations

import numpy as np


def logits(x, router):
    """(x router^T, sums of |terms|)."""
    return x @ router.T, np.abs(x) @ np.abs(router).T


def select(score32, bias32, k):
    """Top-k ids of float32 score + bias: above the k-th largest key ascending, then its equals ascending."""
    key = (score32 + bias32).astype(np.float32)
    out = np.zeros((key.shape[0], k), np.int64)
    for t, row in enumerate(key):
        kth = np.sort(row)[::-1][k - 1]
        above = np.flatnonzero(row > kth)
        out[t] = np.concatenate([above, np.flatnonzero(row == kth)])[:k]
    return out


def probs(score, idx, scaling):
    p = np.take_along_axis(score, idx, 1)
    p = p / (p.sum(1, keepdims=True) + 1e-20)
    return p if scaling is None else p * scaling


def experts(x, wg, wu, wd, idx, p):
    """(y, sum of |terms| of y) in float64; the weights are arrays or functions of the expert."""
    get = lambda w, e: (w(e) if callable(w) else w[e])  # noqa: E731
    d = x.shape[1]
    y, mag = np.zeros((x.shape[0], d)), np.zeros((x.shape[0], d))
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        hg, hu = x[t] @ get(wg, e).T, x[t] @ get(wu, e).T
        h = hg / (1.0 + np.exp(-hg)) * hu * p[t, j][:, None]
        y[t] += h @ get(wd, e).T
        mag[t] += np.abs(h) @ np.abs(get(wd, e)).T
    return y, mag
