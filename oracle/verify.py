"""Verification of drafted tokens, one sequence at a time in fp64."""
from __future__ import annotations

import numpy as np

__all__ = ["verify_drafts"]


def verify_drafts(target, draft_tokens, u_accept, u_next, draft_probs=None, n_drafts=None):
    """numpy arrays shaped as the library's; returns (tokens [S, K+1], accepted [S]) int32."""
    S, K1, V = target.shape
    K = K1 - 1
    tokens = np.full((S, K1), -1, np.int32)
    accepted = np.zeros(S, np.int32)
    for s in range(S):
        n = K if n_drafts is None else min(max(int(n_drafts[s]), 0), K)
        a = 0
        while a < n:
            x = int(draft_tokens[s, a])
            if not 0 <= x < V:
                break
            q = 1.0 if draft_probs is None else float(draft_probs[s, a, x])
            if not float(u_accept[s, a]) * q < float(target[s, a, x]):
                break
            tokens[s, a] = x
            a += 1
        p = np.where(target[s, a] > 0, target[s, a], 0).astype(np.float64)
        r = p
        if a < n:
            q = np.zeros(V)
            if draft_probs is not None:
                q = draft_probs[s, a].astype(np.float64)
            elif 0 <= int(draft_tokens[s, a]) < V:
                q[int(draft_tokens[s, a])] = np.inf
            r = np.where(p > q, p - q, 0)
            if not r.sum() > 0:
                r = p
        c = np.cumsum(r)
        accepted[s] = a
        if c[-1] > 0:
            first = np.nonzero(c > float(u_next[s]) * c[-1])[0]
            tokens[s, a] = first[0] if len(first) else np.nonzero(r > 0)[0][-1]
    return tokens, accepted
