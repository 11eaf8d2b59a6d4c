"""Sampling for whole batches at full vocabularies (tpa_sample_tokens): 4, 2 and 1 CTAs a row, among them rows of more tokens a CTA than
the histograms' 32-bit halves have room for.  Against fp64 on the device.

Borders are off by 2^-29 of the whole, top_p's by 2^-28 more; each is held to 2^-27.  A token whose run ends that near to top_p may be kept or not: its
weight is added to what the draw may be off by.  Log-probabilities: 2^-23 + 2^-22 of themselves, and what such a token makes of the kept sum."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _kept(x, temperature, top_p, off):
    """Weights of what top_p keeps, with its target off by a share of itself."""
    w = ((x - x.amax(1, keepdim=True)) / float(np.float32(temperature))).exp()
    if top_p == 1:
        return w
    at = torch.sort(x, dim=1, descending=True, stable=True).indices
    run = w.gather(1, at)
    before = run.cumsum(1) - run
    run[before >= float(np.float32(top_p)) * (1 + off) * run.sum(1, keepdim=True)] = 0
    return torch.zeros_like(w).scatter_(1, at, run)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(76, 151936), (151, 151936), (301, 151936), (512, 151936), (303, 70001)])
@pytest.mark.parametrize("temperature,top_p", [(1.0, 1.0), (1.0, 0.9), (1.3, 0.97), (4.0, 0.5)])
def test_batches(tpa, n, v, dtype, temperature, top_p):
    g = torch.Generator(device="cuda").manual_seed(n + v)
    x = 2.5 * torch.randn((n, v), generator=g, device="cuda")
    x.scatter_add_(1, torch.randint(0, v, (n, 24), generator=g, device="cuda"), 4 + 10 * torch.rand((n, 24), generator=g, device="cuda"))
    x[1::7] = (2 * x[1::7]).round() / 2         # many equal
    x[2::7, v // 5:] = -torch.inf                # most masked
    x = x.to(dtype)
    u = torch.rand(n, generator=g, device="cuda")
    u[:4] = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 2.0 ** -24])
    t, l = torch.full((n,), -7777, dtype=torch.int32, device="cuda"), torch.full((n,), 7777.0, device="cuda")
    tpa.sample_tokens(x, u, temperature, 0, top_p, out=(t, l))
    tpa.sync_status()
    for rows in range(0, n, 64):                 # (64 rows of 151936 in fp64: 78 MB a tensor)
        some = slice(rows, rows + 64)
        most, least = (_kept(x[some].double(), temperature, top_p, s * 2.0 ** -27) for s in (1, -1))
        unsure = (most - least).sum(1)
        at = t[some].long()[:, None]
        assert ((at >= 0) & (at < v)).all()
        mine = most.gather(1, at)[:, 0]
        sums = most.cumsum(1)
        whole, upper = sums[:, -1], sums.gather(1, at)[:, 0]
        limit = u[some].double() * whole
        slack = 2.0 ** -27 * whole + unsure
        assert (mine > 0).all()
        assert (upper - mine <= limit + slack).all() and (limit <= upper + slack).all()
        want = (mine / whole).log()
        assert ((l[some].double() - want).abs() <= 2.0 ** -23 + 2.0 ** -22 * want.abs() + unsure / whole + 2.0 ** -27).all()
