"""Head norms, rotary positions and their gradient in fp64, from the formulas:
y = R(p) (x r w), r = (mean x^2 + eps)^(-1/2)."""
from __future__ import annotations

import torch

__all__ = ["rope_angles", "norm_rope", "norm_rope_grad"]


def rope_angles(n_positions: int, rot_dim: int, base: float = 10000.0, inv_freq=None, scale: float = 1.0):
    """cos | sin of position x frequency, fp64 [n_positions, rot_dim]."""
    f = (torch.tensor([base ** (-2.0 * j / rot_dim) for j in range(rot_dim // 2)], dtype=torch.float64)
         if inv_freq is None else torch.as_tensor(inv_freq, dtype=torch.float64))
    a = torch.arange(n_positions, dtype=torch.float64)[:, None] * f
    return scale * torch.cat([torch.cos(a), torch.sin(a)], 1)


def _pairs(d_rot: int, interleaved: bool):
    j = torch.arange(d_rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + d_rot // 2)


def _turn(x, row, interleaved: bool, sign: float):
    """x [n, h, d] turned pair by pair by the angles of row [n, rot]."""
    rot = row.shape[1]
    c, s = row[:, None, :rot // 2], sign * row[:, None, rot // 2:]
    a, b = _pairs(rot, interleaved)
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _pair_size(x, rot: int, interleaved: bool):
    size = x.abs()
    a, b = _pairs(rot, interleaved)
    both = x[..., a].abs() + x[..., b].abs()
    size[..., a] = both
    size[..., b] = both
    return size


def _rstd(x, eps):
    return (x.square().mean(-1, keepdim=True) + eps) ** -0.5


def norm_rope(x, w, row, eps: float, interleaved: bool):
    """x [n, h, d], w [d] or None, row [n, rot] (None: no rotation) -> y fp64,
    and for each value the magnitudes that it was summed from."""
    x = x.double()
    if w is not None:
        x = x * _rstd(x, eps) * w.double()
    if row is None:
        return x, x.abs()
    row = row.double()
    return _turn(x, row, interleaved, 1.0), _pair_size(x, row.shape[1], interleaved)


def norm_rope_grad(g, x, w, row, eps: float, interleaved: bool):
    """Gradients of <g, y>: dx, dw, and the magnitudes that each was summed from."""
    g, row = g.double(), row.double()
    z = _turn(g, row, interleaved, -1.0)
    zs = _pair_size(g, row.shape[1], interleaved)
    if w is None:
        return z, None, zs, None
    x, w = x.double(), w.double()
    r = _rstd(x, eps)
    h = x * r
    dw = (z * h).sum((0, 1))
    dx = r * (z * w - h * (z * w * h).mean(-1, keepdim=True))
    size = r * (zs * w.abs() + h.abs() * (zs * w.abs() * h.abs()).mean(-1, keepdim=True))
    return dx, dw, size, (zs * h.abs()).sum((0, 1))
