"""Draws at the ends of u and at the borders between a row's parts (tpa_sample_tokens), at vocabularies of
real size and on every number of CTAs a row.  Against fp64 sums on the device.

A weight is off by at most 2^-29 of itself and a unit, 2^-(61 - log2 vocab) of the row's largest (log2 rounded up), and a running sum by the
units of the tokens in it, two each at most where the row has no cut (the sum is kept in units that grow with the running maximum).  So a draw's
borders are off by 2^-28 of the sum and 2 vocab units; for u = 1 the tokens behind the one drawn weigh a unit
each at most.  Log-probabilities as in test_gpu_sample.py, next to the cut-off 3 2^-24 (64 + 44)."""
import math

import numpy as np
import pytest
import torch

from _pipeline import check_guards, guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _rows(n, v, dtype, order):
    g = torch.Generator(device="cuda").manual_seed(n + v)
    x = 2.5 * torch.randn((n, v), generator=g, device="cuda")
    at = torch.randint(0, v, (n, 24), generator=g, device="cuda")
    x.scatter_add_(1, at, 4 + 10 * torch.rand((n, 24), generator=g, device="cuda"))
    if order == "rising":
        x = 2 * x.sort(1).values
    elif order == "steps":   # every run of 500 tokens rises
        x[:, :v // 500 * 500] = x[:, :v // 500 * 500].view(n, -1, 500).sort(2).values.view(n, -1)
    return x.to(dtype)


def _draw(tpa, x, u, **kw):
    """Tokens and log-probabilities, in tensors that hold neither before."""
    bt, t = guarded((len(x),), torch.int32)
    bl, l = guarded((len(x),), torch.float32)
    t.fill_(-7777)
    l.fill_(7777.0)
    tpa.sample_tokens(x, u, out=(t, l), **kw)
    check_guards(bt, "tokens")
    check_guards(bl, "logp")
    assert (t != -7777).all() and (l != 7777.0).all(), f"rows left as they were: {(t == -7777).nonzero()[:, 0].tolist()}"
    return t, l


def _check(x, u, t, l, kept=None):
    n, v = x.shape
    w = (x.double() - x.double().amax(1, keepdim=True)).exp()
    if kept is not None:
        w = torch.where(kept, w, 0.0)
    assert ((t >= 0) & (t < v)).all()
    at = t.long()[:, None]
    mine = w.gather(1, at)[:, 0]
    assert (mine > 0).all()
    sums = w.cumsum(1)
    whole, upper = sums[:, -1], sums.gather(1, at)[:, 0]
    unit = 2.0 ** -(61 - math.ceil(math.log2(v)))
    slack = 2.0 ** -28 * whole + 2 * v * unit
    limit = u.double() * whole
    assert (upper - mine <= limit + slack).all() and (limit <= upper + slack).all()
    behind = torch.where(torch.arange(v, device="cuda") > at, w, 0.0).amax(1)
    assert (behind[u >= 1] <= unit * (1 + 2.0 ** -20)).all()
    assert ((l.double() - (mine / whole).log()).abs() <= 3 * 2.0 ** -24 * (64 + 44)).all()


ENDS = (0.0, 2.0 ** -149, 2.0 ** -24, 0.25, 0.5, 1 - 2.0 ** -23, 1 - 2.0 ** -24, 1.0)


@pytest.mark.parametrize("order", ["any", "rising", "steps"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(20, 151936), (90, 151937), (160, 50001), (310, 32000), (20, 5003)])   # 8, 4, 2, 1, 1 or 2 CTAs
def test_ends_without_a_cut(tpa, n, v, dtype, order):
    x = _rows(n, v, dtype, order)
    each = torch.ones(n, device="cuda")
    for value in ENDS:
        u = torch.full((n,), value, device="cuda")
        _check(x, u, *_draw(tpa, x, u))
        _check(x, u, *_draw(tpa, x, u, temperature=each))   # the rows as those with cuts are gone through
    u = torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    _check(x, u, *_draw(tpa, x, u))
    tpa.sync_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(20, 151936), (160, 50001), (310, 32000)])
def test_ends_with_cuts(tpa, n, v, dtype):
    x = _rows(n, v, dtype, "any")
    top, at = torch.sort(x, dim=1, descending=True, stable=True)
    first = torch.zeros_like(x, dtype=torch.bool).scatter_(1, at[:, :50], True)
    some = (x.double() - x.double().amax(1, keepdim=True)).exp() >= float(np.float32(1e-3))
    index = torch.arange(v, device="cuda")
    for value in ENDS:
        u = torch.full((n,), value, device="cuda")
        for kept, kw in ((first, dict(top_k=50)), (some, dict(min_p=1e-3)), (first & some, dict(top_k=50, min_p=1e-3))):
            t, l = _draw(tpa, x, u, **kw)
            _check(x, u, t, l, kept)
            if value == 0.0:
                assert torch.equal(t.long(), torch.where(kept, index, v).amin(1))
            if value == 1.0:
                assert torch.equal(t.long(), torch.where(kept, index, -1).amax(1))
    tpa.sync_status()


def _below_a_unit(parts):
    """A row of 2^24 logits whose parts (64, one a warp) hold nothing but, in `parts`, 2^18 - 1 tokens of 0.9 units of the largest weight, 2^38 units, and
    behind them one of that weight."""
    v = 1 << 24
    x = torch.full((v,), -math.inf, device="cuda")
    for p in parts:
        x[p << 18:(p + 1) << 18] = (math.log2(0.9) - 38) * math.log(2)
        x[(p + 1 << 18) - 1] = 0.0
    return x


def test_ends_of_parts_that_begin_with_less_than_a_unit(tpa):
    # 0.9 units 2^18 - 1 times: 235929 units; u's steps next to 1 are 2^14 units of one such part, next to 1/2 of two
    last = _below_a_unit([63])[None].expand(7, -1).contiguous()
    u = torch.tensor([1.0] + [1 - i * 2.0 ** -24 for i in range(1, 7)], device="cuda")
    t, l = _draw(tpa, last, u)
    assert (t == (1 << 24) - 1).all()
    assert (l.abs() <= 2.0 ** -20 + 2.0 ** -23).all()   # 235929 of 2^38 units
    two = _below_a_unit([20, 63])[None].expand(14, -1).contiguous()
    u = torch.tensor([0.5 - i * 2.0 ** -25 for i in range(1, 15)], device="cuda")
    t, l = _draw(tpa, two, u)
    assert (t == (21 << 18) - 1).all()
    assert ((l - math.log(0.5)).abs() <= 2.0 ** -20 + 2.0 ** -23).all()
    tpa.sync_status()
