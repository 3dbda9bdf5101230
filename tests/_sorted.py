"""Routings for the tests of the sorted-row operators, and their definitions in
64 bits (numpy)."""
from __future__ import annotations

import numpy as np

W_SCALE = 1.5


def routing(T, k, E, seed, drop=0.0, only=None):
    """(logits, ids, w, offsets, row_src, row_dst) of T tokens: top-k of random
    logits, each token's tail pruned with probability `drop` a slot, whole
    tokens among them; `only`: every id from this range of experts."""
    g = np.random.default_rng(seed)
    logits = g.standard_normal((T, E)).astype(np.float32)
    pool = logits if only is None else np.where(np.isin(np.arange(E), only), logits, -np.inf)
    ids = np.argsort(-pool, axis=1, kind="stable")[:, :k].astype(np.int32)
    m = (g.random((T, k)) >= drop).sum(1)
    ids[np.arange(k)[None, :] >= m[:, None]] = -1
    w = np.where(ids >= 0, g.random((T, k)) + 0.1, 0).astype(np.float32)
    flat = np.where(ids.reshape(-1) < 0, E, ids.reshape(-1))
    row_src = np.argsort(flat, kind="stable").astype(np.int32)
    row_dst = np.empty(T * k, np.int32)
    row_dst[row_src] = np.arange(T * k)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])]).astype(np.int32)
    row_dst[flat == E] = -1
    return logits, ids, w, offsets, row_src, row_dst


def combine64(y, w, row_dst, T, k):
    """(sum, sum of absolute values) of w * y over the filled slots."""
    out = np.zeros((T, y.shape[1]))
    mag = np.zeros_like(out)
    for j in range(k):
        d = row_dst.reshape(T, k)[:, j]
        on = d >= 0
        term = y[d[on]] * (1.0 if w is None else w[on, j, None].astype(np.float64))
        out[on] += term
        mag[on] += np.abs(term)
    return out, mag


def route_weights64(l, ids):
    """The router's weights of the kept slots, in 64 bits."""
    kept = ids >= 0
    s = np.where(kept, np.sqrt(np.logaddexp(0, np.take_along_axis(l, np.maximum(ids, 0), 1))), 0)
    total = s.sum(1, keepdims=True)
    return W_SCALE * s / np.where(total > 0, total, 1)


def route_grad64(logits, ids, dw):
    """(dlogits, sum of the absolute values of its terms)."""
    l = logits.astype(np.float64)
    kept = ids >= 0
    at = np.maximum(ids, 0)
    lk = np.take_along_axis(l, at, 1)
    s = np.where(kept, np.sqrt(np.logaddexp(0, lk)), 0)
    total = s.sum(1)
    grad, mag = np.zeros_like(l), np.zeros_like(l)
    for t, j in zip(*np.nonzero(kept)):
        slope = W_SCALE / total[t] ** 2 / (1 + np.exp(-lk[t, j])) / (2 * s[t, j])
        on = kept[t]
        grad[t, at[t, j]] += slope * (s[t][on] * (dw[t, j] - dw[t][on])).sum()
        mag[t, at[t, j]] += slope * (s[t][on] * (abs(dw[t, j]) + np.abs(dw[t][on]))).sum()
    return grad, mag
