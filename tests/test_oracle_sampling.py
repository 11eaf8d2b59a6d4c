"""Pins of the oracles of a sampling step's operators (CPU): kept sets and draws of small rows worked out by
hand or by brute force, distributions, trees whose answers are plain, and a cache's pages under random use."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle.draft import accept, attend_tree, masks
from oracle.pages import Pool
from oracle.paged import attend_sequence
from oracle.sample import kept_weights, sample_tokens

LOG = [math.log(p) for p in (0.1, 0.4, 0.1, 0.25, 0.15)]   # weights 0.25, 1, 0.25, 0.625, 0.375 of the largest


@pytest.mark.parametrize("kw,kept", [
    (dict(), [0, 1, 2, 3, 4]),
    (dict(top_k=1), [1]),
    (dict(top_k=2), [1, 3]),
    (dict(top_k=4), [0, 1, 3, 4]),           # of two equal ones the first
    (dict(top_k=9), [0, 1, 2, 3, 4]),
    (dict(top_p=0.0), [1]),
    (dict(top_p=0.39), [1]),
    (dict(top_p=0.41), [1, 3]),
    (dict(top_p=0.64), [1, 3]),
    (dict(top_p=0.66), [1, 3, 4]),
    (dict(top_p=0.89), [0, 1, 3, 4]),
    (dict(min_p=0.3), [1, 3, 4]),
    (dict(min_p=0.5), [1, 3]),
    (dict(min_p=1.0), [1]),
    (dict(top_k=3, top_p=0.79), [1, 3]),     # of 0.8 that top_k leaves: 0.65 / 0.8 = 0.8125
    (dict(top_k=3, top_p=0.82), [1, 3, 4]),
    (dict(top_p=0.95, min_p=0.3), [1, 3, 4]),
])
def test_kept_sets_by_hand(kw, kept):
    w = kept_weights(LOG, 1.0, **kw)
    assert np.nonzero(w)[0].tolist() == kept
    assert np.allclose(w[kept], np.exp(LOG)[kept] / 0.4, rtol=1e-12)


def test_temperature():
    assert np.allclose(kept_weights(LOG, 0.5), (np.exp(LOG) / 0.4) ** 2, rtol=1e-12)
    assert np.nonzero(kept_weights([1.0, 3.0, 3.0], 0.0))[0].tolist() == [1]
    assert np.nonzero(kept_weights([-np.inf, np.nan, -4.0], 1.0))[0].tolist() == [2]
    assert not kept_weights([-np.inf, np.nan], 1.0).any()
    assert np.nonzero(kept_weights([np.inf, 5.0, np.inf], 0.0))[0].tolist() == [0]


@pytest.mark.parametrize("kw", [dict(), dict(top_k=3), dict(top_p=0.66), dict(min_p=0.3), dict(top_k=4, top_p=0.9, min_p=0.26)])
def test_draws_have_the_kept_distribution(kw):
    # every u of a fine comb: frequencies within the comb's pitch
    n = 20000
    u = (np.arange(n) + 0.5) / n
    args = {**dict(top_k=0, top_p=1.0, min_p=0.0), **kw}
    t, logp = sample_tokens(np.tile(LOG, (n, 1)), u, np.ones(n), *(np.full(n, args[k]) for k in ("top_k", "top_p", "min_p")))
    w = kept_weights(LOG, 1.0, **kw)
    p = w / w.sum()
    assert (np.abs(np.bincount(t, minlength=5) / n - p) <= 1 / n + 1e-12).all()
    assert np.allclose(np.exp(logp), p[t], rtol=1e-12)
    assert (np.diff(t) >= 0).all()


def test_masks_and_positions_by_hand():
    #   0 - 1 - 3 - 4, 0 - 2, 5 alone
    pos, words = masks([-1, 0, 0, 1, 3, -1], 10, 1)
    assert pos == [10, 11, 11, 12, 13, 10]
    assert [w[0] for w in words] == [0b1, 0b11, 0b101, 0b1011, 0b11011, 0b100000]
    assert [w[0] for w in masks([-1, 0, 0, 1, 3, -1], 10, 1, window=2)[1]] == [0b1, 0b11, 0b101, 0b1010, 0b11000, 0b100000]
    chain = masks(list(range(-1, 39)), 0, 2)[1]
    assert chain[39] == [-1, 0xff] and chain[31] == [-1, 0] and chain[30] == [2 ** 31 - 1, 0]


def test_masks_are_the_ancestors():
    r = np.random.default_rng(0)
    for _ in range(30):
        n = int(r.integers(1, 70))
        parents = [int(r.integers(-1, i)) if i else -1 for i in range(n)]
        up = np.zeros((n, n), bool)
        for i, p in enumerate(parents):
            if p >= 0:
                up[i, p] = True
        reach = np.linalg.matrix_power((up + np.eye(n)).astype(object), n) > 0   # paths of up to n links
        pos, words = masks(parents, 5, 3)
        got = np.array([[w[j // 32] >> (j % 32) & 1 for j in range(n)] for w in words], bool)
        assert (got == reach).all()
        assert pos == [4 + int(x) for x in reach.sum(1)]


@pytest.mark.parametrize("most", [1, 2, 4])
def test_accepted_paths_by_brute_force(most):
    # all parents, drafted and sampled tokens (of two) of a tree of four: the path is the longest chain of rows, each the
    # first fitting child of the one before
    for parents in itertools.product([-1], [0], range(-1, 2), range(-1, 3)):
        for drafted in itertools.product([0], *[range(2)] * 3):
            for sampled in itertools.product(range(-1, 2), repeat=4):
                def fits(r, j):
                    return parents[j] == r and drafted[j] == sampled[r] and sampled[r] >= 0
                chains = [c for n in range(1, 5) for c in itertools.combinations(range(4), n) if c[0] == 0 and all(
                    fits(a, b) and not any(fits(a, j) for j in range(b)) for a, b in zip(c, c[1:]))]
                path = list(max(chains, key=len))[:most]
                assert accept(parents, drafted, sampled, most) == (path, [sampled[r] for r in path])
    assert accept([], [], [], 3) == ([], [])


def test_paths_are_distributed_as_the_policy():
    # a policy that draws b with 0.3 behind anything: the first two tokens behind a root whose children are drafted
    r = np.random.default_rng(1)
    n, counts = 20000, np.zeros((2, 2))
    for _ in range(n):
        sampled = (r.random(5) < 0.3).astype(int).tolist()
        path, tokens = accept([-1, 0, 1, 0, 3], [0, 0, 0, 1, 1], sampled, 5)
        counts[tokens[0], tokens[1]] += 1          # (both tokens are drafted: the path has two rows at least)
    want = np.outer([0.7, 0.3], [0.7, 0.3]) * n
    assert (np.abs(counts - want) <= 5 * np.sqrt(want)).all()


def test_attention_under_a_chains_mask_is_the_causal_one():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(s, generator=g) for s in ((7, 4, 64), (30, 2, 64), (30, 2, 64)))
    o, lse, _ = attend_tree(q, k, v, torch.arange(30)[None] <= torch.arange(23, 30)[:, None])
    want = attend_sequence(q, k, v)
    assert (o - want[0]).abs().max() < 1e-12 and (lse - want[1]).abs().max() < 1e-12
    o, lse, size = attend_tree(q, k, v, torch.zeros((7, 30), dtype=torch.bool))
    assert (o == 0).all() and torch.isneginf(lse).all() and (size == 0).all()


def test_pages_under_random_use():
    r = np.random.default_rng(4)
    pool = Pool(40, 8, 16)
    short = 0
    for _ in range(400):
        before = [list(x) for x in pool.rows]
        if r.random() < 0.5:
            lens = [int(x) * int(r.random() < 0.7) for x in r.integers(0, 140, 8)]
            left = pool.resize(lens)
            need = [-(-n // 16) for n in lens]
            assert [len(x) for x in pool.rows] == (need if left >= 0 else [min(n, len(b)) for n, b in zip(need, before)])
            if left < 0:
                pool.resize([len(x) * 16 for x in pool.rows])
        else:
            rows = [int(x) for x in r.permutation(8)]
            src, dst = [rows[0], rows[0], rows[1]], rows[2:5]
            left, copies = pool.fork(src, dst)
            for s, d in zip(src, dst):
                whole, part = divmod(pool.lens[s], 16)
                if left < 0:
                    assert pool.rows[d] == [] and pool.lens[d] == 0
                else:
                    assert pool.lens[d] == pool.lens[s] and pool.rows[d][:whole] == pool.rows[s][:whole]
                    assert len(pool.rows[d]) == whole + (part > 0)
                    if part:
                        assert (pool.rows[s][whole], pool.rows[d][whole], part) in copies
        short += left < 0
        used = [p for x in pool.rows for p in x]
        assert pool.refs == [used.count(p) for p in range(40)]
        assert all(len(set(x)) == len(x) for x in pool.rows)
        assert left < 0 or left == pool.refs.count(0)
    assert short > 0  # (it has run short at all)
