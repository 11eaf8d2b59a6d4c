"""Pins of the fp64 oracles of the policy's operators (CPU): the rotation keeps
lengths and depends on distances, the gradient agrees with differences, a drawn
token has the probability it should."""
import numpy as np
import pytest
import torch

from oracle.paged import attend_sequence
from oracle.rope import norm_rope, norm_rope_grad, rope_angles
from oracle.verify import verify_drafts


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance(interleaved):
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn((1, 1, 64), generator=g), torch.randn((1, 1, 64), generator=g)
    t = rope_angles(300, 64)

    def dot(i, j):
        a, _ = norm_rope(q, None, t[i:i + 1], 0.0, interleaved)
        b, _ = norm_rope(k, None, t[j:j + 1], 0.0, interleaved)
        assert abs(a.norm() - q.double().norm()) < 1e-12
        return float((a * b).sum())

    assert abs(dot(7, 3) - dot(207, 203)) < 1e-10
    assert abs(dot(7, 3) - dot(7, 4)) > 1e-3


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 32, 64])
def test_gradient_against_differences(interleaved, rot):
    g = torch.Generator().manual_seed(2)
    x, dy = (torch.randn((3, 2, 64), generator=g, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.3 * torch.randn(64, generator=g, dtype=torch.float64)
    row = rope_angles(9, rot)[[0, 4, 8]]
    dx, dw, _, _ = norm_rope_grad(dy, x, w, row, 1e-6, interleaved)

    def f(x_, w_):
        return float((norm_rope(x_, w_, row, 1e-6, interleaved)[0] * dy).sum())

    e = 1e-6
    for i in ((0, 0, 0), (1, 1, 15), (2, 0, 16), (2, 1, 63), (0, 1, 40)):
        d = torch.zeros_like(x)
        d[i] = e
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * e) - dx[i]) < 1e-7
    for i in (0, 8, 33, 63):
        d = torch.zeros_like(w)
        d[i] = e
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * e) - dw[i]) < 1e-7


def test_verified_tokens_follow_the_target():
    # 40000 sequences of one draft each: the first token's frequencies are the target's (5 standard deviations)
    rng = np.random.default_rng(3)
    V, S = 5, 40000
    p = np.array([0.1, 0.4, 0.2, 0.25, 0.05], np.float32)
    q = np.array([0.4, 0.1, 0.3, 0.1, 0.1], np.float32)
    x = rng.choice(V, size=(S, 1), p=q.astype(np.float64) / q.astype(np.float64).sum()).astype(np.int32)
    target = np.broadcast_to(p, (S, 2, V))
    tokens, n = verify_drafts(target, x, rng.random((S, 1), np.float32), rng.random(S, np.float32),
                              np.broadcast_to(q, (S, 1, V)))
    share = np.bincount(tokens[:, 0], minlength=V) / S
    assert np.all(np.abs(share - p) < 5 * np.sqrt(p * (1 - p) / S))
    assert abs(n.mean() - np.minimum(p, q).sum()) < 5 * 0.5 / np.sqrt(S)


def test_verify_by_hand():
    target = np.array([[[0.5, 0.5, 0.0], [0.0, 1.0, 0.0], [0.25, 0.25, 0.5]]], np.float32)
    x = np.array([[0, 1]], np.int32)
    u = np.array([[0.4, 0.9]], np.float32)
    assert verify_drafts(target, x, u, np.array([0.5], np.float32))[0].tolist() == [[0, 1, 2]]
    assert verify_drafts(target, x, u, np.array([0.49], np.float32))[0].tolist() == [[0, 1, 1]]
    # the second drafted token is turned down, and what is left is all on token 1
    t, n = verify_drafts(target, np.array([[0, 2]], np.int32), u, np.array([0.0], np.float32))
    assert t.tolist() == [[0, 1, -1]] and n.tolist() == [1]
    # the first is turned down: what is left without it is token 0
    t, n = verify_drafts(target, np.array([[1, 1]], np.int32), np.array([[0.6, 0.0]], np.float32),
                         np.array([0.3], np.float32))
    assert t.tolist() == [[0, -1, -1]] and n.tolist() == [0]
    # a draft with all of the target's weight that is turned down by u = 1: the target itself is drawn from
    t, n = verify_drafts(np.array([[[0.0, 1.0], [1.0, 0.0]]], np.float32), np.array([[1]], np.int32),
                         np.array([[1.0]], np.float32), np.array([0.5], np.float32))
    assert t.tolist() == [[1, -1]] and n.tolist() == [0]


@pytest.mark.parametrize("n,kv,window", [(1, 1, 0), (5, 9, 0), (4, 12, 3), (6, 4, 0), (3, 0, 0), (2, 30, 1)])
def test_attention_over_a_cache_against_the_library(n, kv, window):
    """The last n tokens of kv, causal at the end, grouped heads; rows before the first cached token see nothing."""
    g = torch.Generator().manual_seed(n + kv)
    q = torch.randn((n, 6, 16), generator=g, dtype=torch.float64)
    k, v = (torch.randn((kv, 2, 16), generator=g, dtype=torch.float64) for _ in range(2))
    o, lse, size = attend_sequence(q, k, v, window)
    i, j = torch.arange(kv - n, kv)[:, None], torch.arange(kv)[None]
    seen = (j <= i) & (j > i - (window or kv + 1))
    rows = seen.any(1)
    assert (o[~rows] == 0).all() and torch.isneginf(lse[~rows]).all() and torch.isfinite(lse[rows]).all()
    if rows.any():
        want = torch.nn.functional.scaled_dot_product_attention(
            q[rows].transpose(0, 1), k.repeat_interleave(3, 1).transpose(0, 1), v.repeat_interleave(3, 1).transpose(0, 1),
            attn_mask=seen[rows]).transpose(0, 1)
        assert (o[rows] - want).abs().max() < 1e-13 and (size[rows] >= o[rows].abs() - 1e-13).all()
        x = torch.einsum("nhd,hkd->nhk", q[rows], k.repeat_interleave(3, 1).transpose(0, 1)) / 4.0
        p = (x - lse[rows][..., None]).exp() * seen[rows][:, None]
        assert (p.sum(-1) - 1).abs().max() < 1e-13
