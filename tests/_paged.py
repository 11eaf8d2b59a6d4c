"""Seeded batches over a paged cache for the tests of the sampling side."""
from __future__ import annotations

import numpy as np
import torch


class Batch:
    """Sequences of q_lens new tokens and kv_lens cached ones (the new ones
    included) on shuffled pages of a cache of random values; ``extra`` rows of
    padding behind the last sequence."""

    def __init__(self, q_lens, kv_lens, hq, hkv, d, page, seed, extra=0, spare=3, device="cuda"):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens_list = list(q_lens), list(kv_lens)
        self.hq, self.hkv, self.d, self.page = hq, hkv, d, page
        need = [-(-n // page) for n in kv_lens]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages).tolist()
        width = max(1, max(need, default=1))
        rows, at = [], 0
        for n in need:
            rows.append(order[at:at + n] + [-1] * (width - n))  # entries past the sequence are not looked at
            at += n
        self.rows = rows
        self.total = sum(q_lens)
        n = self.total + extra
        self.pages = torch.tensor(rows, dtype=torch.int32).view(len(rows), width).to(device)
        self.offsets = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32).to(device)
        self.kv_lens = torch.tensor(kv_lens, dtype=torch.int32).to(device)
        bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(device)  # noqa: E731
        self.k_cache, self.v_cache = bf(self.n_pages, hkv, page, d), bf(self.n_pages, hkv, page, d)
        self.q, self.k, self.v = bf(n, hq, d), bf(n, hkv, d), bf(n, hkv, d)

    @property
    def cache(self):
        return self.k_cache, self.v_cache, self.pages, self.offsets, self.kv_lens

    def places(self):
        """(sequence, position) of every new token, int64 on the CPU."""
        s = np.repeat(np.arange(len(self.q_lens)), self.q_lens)
        p = np.concatenate([np.arange(b - a, b) for a, b in zip(self.q_lens, self.kv_lens_list)] or [[]])
        return torch.from_numpy(s.astype(np.int64)), torch.from_numpy(p.astype(np.int64))

    def slots(self):
        """(page, slot) of every new token."""
        s, p = self.places()
        return self.pages.cpu().long()[s, p // self.page], p % self.page

    def sequence(self, s, cache):
        """Cached rows [kv_len, hkv, d] of sequence s, fp64 on the CPU."""
        j = torch.arange(self.kv_lens_list[s])
        page = torch.tensor(self.rows[s], dtype=torch.long)[j // self.page]
        return cache.cpu()[page, :, j % self.page].double()
