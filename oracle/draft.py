"""Drafted trees: positions, masks, the path of the sampled tokens, and attention under masks, one sequence at a time."""
from __future__ import annotations

import math

import torch

__all__ = ["accept", "attend_tree", "masks"]


def masks(parents, base: int, words: int, window: int = 0):
    """parents: a sequence's list.  Returns positions [n] and mask words [n][words] (as signed 32-bit numbers)."""
    positions, rows = [], []
    for i in range(len(parents)):
        chain = [i]
        while parents[chain[-1]] >= 0:
            chain.append(parents[chain[-1]])
        positions.append(base + len(chain) - 1)
        bits = 0
        for j in chain[:window] if window else chain:
            bits |= 1 << j
        w = [bits >> 32 * k & 0xffffffff for k in range(words)]
        rows.append([x - (1 << 32) if x >> 31 else x for x in w])
    return positions, rows


def accept(parents, drafted, sampled, most: int):
    """The rows that stand, at most `most`, and the tokens sampled behind them.  A negative token is nobody's."""
    if not parents or most < 1:
        return [], []
    path = [0]
    while len(path) < most:
        below = [j for j, p in enumerate(parents) if p == path[-1] and drafted[j] == sampled[path[-1]] >= 0]
        if not below:
            break
        path.append(below[0])
    return path, [sampled[r] for r in path]


def attend_tree(q, k, v, seen):
    """q [n, Hq, d], k and v [kv, Hkv, d], seen [n, kv] bool: O, LSE and the sums of
    probabilities times magnitudes, fp64."""
    n, hq, d = q.shape
    kv, hkv, _ = k.shape
    x = torch.einsum("nhgd,khd->nhgk", q.double().view(n, hkv, hq // hkv, d), k.double()) / math.sqrt(d)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    lse = torch.logsumexp(x, -1) if kv else torch.full(x.shape[:-1], -math.inf, dtype=torch.float64)
    some = torch.isfinite(lse)
    p = torch.where(some[..., None], (x - torch.where(some, lse, 0.0)[..., None]).exp(), 0.0)
    o = torch.einsum("nhgk,khd->nhgd", p, v.double())
    size = torch.einsum("nhgk,khd->nhgd", p, v.double().abs())
    return o.reshape(n, hq, d), lse.reshape(n, hq), size.reshape(n, hq, d)
