"""Sampling from logits with temperature, top-k, top-p and min-p, one row at a time in fp64."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["kept_weights", "sample_tokens"]


def kept_weights(x, temperature: float, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """The weights of one row's tokens, 0 for those that are not kept."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    if temperature == 0:
        temperature, top_k = 1.0, 1
    w = np.zeros(len(x))
    top = x.max()
    if top == -np.inf:
        return w
    with np.errstate(over="ignore"):
        each = np.exp((x - top) / temperature)
    order = sorted(range(len(x)), key=lambda v: (-x[v], v))
    order = [v for v in order if x[v] > -np.inf]
    if 0 < top_k < len(x):
        order = order[:top_k]
    if top_p < 1:
        whole, run, n = math.fsum(each[order]), 0.0, 0
        while n == 0 or run < top_p * whole:
            run = math.fsum(each[order[:n + 1]]) if len(order) < 3000 else run + each[order[n]]
            n += 1
            if n == len(order):
                break
        order = order[:n]
    order = [v for v in order if each[v] >= min_p]
    w[order] = each[order]
    return w


def sample_tokens(logits, u, temperature, top_k, top_p, min_p):
    """logits [N, V] fp64; the others [N].  Returns tokens [N] int32 and log-probabilities [N] fp64."""
    n = len(logits)
    tokens, logp = np.full(n, -1, np.int32), np.full(n, np.nan)
    for r in range(n):
        w = kept_weights(logits[r], float(temperature[r]), int(top_k[r]), float(top_p[r]), float(min_p[r]))
        if not w.any():
            continue
        sums = np.cumsum(w)
        past = np.nonzero((sums > float(u[r]) * sums[-1]) & (w > 0))[0]
        tokens[r] = past[0] if len(past) else np.nonzero(w)[0][-1]
        logp[r] = math.log(w[tokens[r]] / sums[-1])
    return tokens, logp
