"""Attention of a sequence's new tokens over its cached keys and values, fp64."""
from __future__ import annotations

import math

import torch

__all__ = ["attend_sequence"]


def attend_sequence(q, k, v, window: int = 0, scale: float | None = None):
    """q [n, Hq, d], k and v [kv, Hkv, d]: the last n of the kv tokens are the
    queries' own.  Returns O [n, Hq, d], LSE [n, Hq] and for each value of O the
    sum of probabilities times magnitudes, all fp64."""
    n, hq, d = q.shape
    kv, hkv, _ = k.shape
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    g = hq // hkv
    q64 = q.double().view(n, hkv, g, d)
    x = torch.einsum("nhgd,khd->nhgk", q64, k.double()) * sc
    pos = torch.arange(kv - n, kv)[:, None]
    j = torch.arange(kv)[None]
    seen = j <= pos
    if window:
        seen &= j > pos - window
    x = x.masked_fill(~seen[:, None, None].to(x.device), -math.inf)
    lse = torch.logsumexp(x, -1) if kv else torch.full(x.shape[:-1], -math.inf, dtype=torch.float64)
    p = torch.where(torch.isfinite(lse)[..., None], (x - torch.where(torch.isfinite(lse), lse, 0.0)[..., None]).exp(), 0.0)
    o = torch.einsum("nhgk,khd->nhgd", p, v.double())
    size = torch.einsum("nhgk,khd->nhgd", p, v.double().abs())
    return o.reshape(n, hq, d), lse.reshape(n, hq), size.reshape(n, hq, d)
