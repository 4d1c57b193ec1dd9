"""Sampling by its definition, one row at a time, in 64 bits (numpy): what
ssc_sample_rows is tested against."""
from __future__ import annotations

import numpy as np


def sample_row(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, kept, logprob) of one row of logits (float64 values)."""
    x = np.where(np.isnan(x), -np.inf, x)
    if np.any(x == np.inf):  # no token beside +infinity
        x = np.where(x == np.inf, 0.0, -np.inf)
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if order.size == 0:
        return -1, 0, -np.inf
    greedy = not t > 0
    p = 1.0 if np.isnan(p) else p
    m = 0.0 if np.isnan(m) else min(max(m, 0.0), 1.0)
    top = x[order[0]]
    w = np.exp((x[order] - top) / (1.0 if greedy else t))
    n = order.size
    if greedy:
        n = 1
    elif k > 0:
        n = min(n, int(k))
    if p < 1 and not greedy:
        before = np.concatenate([[0.0], np.cumsum(w[:n])[:-1]])
        n = max(1, int((before < p * w[:n].sum()).sum()))
    keep = np.arange(n)[(w[:n] >= m) | (np.arange(n) == 0)]
    kept = keep.size
    by = np.argsort(order[keep])
    index, weight = order[keep][by], w[keep][by]
    run = np.cumsum(weight)
    u = 0.0 if np.isnan(u) else min(max(u, 0.0), 1.0 - 2.0 ** -24)
    at = int(np.searchsorted(run, u * run[-1], side="right"))
    return int(index[at]), kept, float(np.log(weight[at] / run[-1]))


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(tokens, kept, logprobs) of rows; settings as arrays or None."""
    def at(a, r, default):
        return default if a is None else float(a[r])
    rows = [sample_row(logits[r], float(u[r]), at(temperature, r, 1.0), at(top_k, r, 0), at(top_p, r, 1.0), at(min_p, r, 0.0))
            for r in range(len(logits))]
    return (np.array([r[0] for r in rows], np.int32), np.array([r[1] for r in rows], np.int32),
            np.array([r[2] for r in rows], np.float64))
