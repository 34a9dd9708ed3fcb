"""Sampling from logits in 64 bits, from its definition: test infrastructure that shares nothing with the
CUDA path."""
from __future__ import annotations

import numpy as np


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, margin) of one row: margin is how near, in units of the weights' sums, the
    nearest decision is to falling the other way (u to an end of its token's interval, a running sum
    to top_p's share)."""
    x = np.asarray(logits, np.float64) + 0.0
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return -1, -np.inf, 1.0
    if not temperature > 0:
        return int(np.argmax(x)), 0.0, 1.0
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.exp((x - top) / temperature)
    w[x == top] = 1.0
    w[np.isnan(w)] = 1.0 if temperature == np.inf else 0.0
    w[x == -np.inf] = 0.0
    if top == np.inf:
        w[x != top] = 0.0
    order = np.lexsort((np.arange(len(x)), -x))
    margin = 1.0
    if 0 < top_k < len(x):
        order = order[:top_k]
    if top_p < 1:
        upto = np.cumsum(w[order])
        reach = max(top_p, 0.0) * upto[-1]
        n = int((upto < reach).sum()) + 1
        order = order[:n]
        margin = min(margin, np.abs(upto - reach).min() / upto[-1])
        if top_p <= 0:
            margin = 1.0
    if min_p > 0:
        order = order[w[order] >= min(min_p, 1.0)]
    stay = np.sort(order)
    stay = stay[w[stay] > 0]
    upto = np.cumsum(w[stay])
    at = min(max(u, 0.0) if u == u else 0.0, 1.0) * upto[-1]
    i = min(int((upto <= at).sum()), len(stay) - 1)
    lo = upto[i - 1] if i else -1.0
    hi = upto[i] if i + 1 < len(stay) else 2 * upto[-1]
    margin = min(margin, (at - lo) / upto[-1], (hi - at) / upto[-1])
    return int(stay[i]), float(np.log(w[stay[i]] / upto[-1])), float(margin)
