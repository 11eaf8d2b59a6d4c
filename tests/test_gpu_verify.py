"""GPU parity of the verification of drafted tokens (tpa_verify_drafts): whole
numbers, equal to the fp64 oracle's.  A draw could differ only where the fp64
running sum is within about 1e-13 of u times the total at a border between two
tokens; no input here is."""
import numpy as np
import pytest
import torch

from oracle.verify import verify_drafts as oracle_verify
from _pipeline import check_guards, guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _probs(g, *shape, near=None):
    x = 2 * torch.randn(shape, generator=g)
    if near is not None:
        x = near + 0.5 * x
    return x, torch.softmax(x, -1)


def _inputs(S, K, V, seed):
    g = torch.Generator().manual_seed(seed)
    logits, p = _probs(g, S, K + 1, V)
    _, q = _probs(g, S, K, V, near=logits[:, :K])
    x = (torch.multinomial(q.reshape(S * K, V), 1, generator=g).view(S, K) if K else torch.zeros((S, 0))).to(torch.int32)
    return p, q, x, torch.rand((S, K), generator=g), torch.rand(S, generator=g), \
        torch.randint(0, K + 1, (S,), generator=g, dtype=torch.int32)


def _check(tpa, p, x, u, un, q=None, n=None):
    S, K1, _ = p.shape
    bt, t = guarded((S, K1), torch.int32)
    ba, a = guarded((S,), torch.int32)
    tpa.verify_drafts(*(z.cuda() for z in (p, x, u, un)), draft_probs=None if q is None else q.cuda(),
                      n_drafts=None if n is None else n.cuda(), out=(t, a))
    check_guards(bt, "tokens")
    check_guards(ba, "accepted")
    want = oracle_verify(*(z.numpy() for z in (p, x, u, un)), None if q is None else q.numpy(),
                         None if n is None else n.numpy())
    assert np.array_equal(a.cpu().numpy(), want[1])
    assert np.array_equal(t.cpu().numpy(), want[0])
    return want


@pytest.mark.parametrize("S,K,V", [(1, 1, 1), (3, 1, 2), (5, 2, 7), (9, 3, 33), (20, 5, 1000), (40, 4, 1001), (3, 8, 4096),
                                   (2, 40, 517), (4, 3, 32000), (6, 2, 151936), (2, 1, 151937), (1, 70, 300)])
@pytest.mark.parametrize("form", ["probs", "ragged", "tokens"])
def test_against_the_oracle(tpa, S, K, V, form):
    p, q, x, u, un, n = _inputs(S, K, V, S + V)
    _check(tpa, p, x, u, un, q if form != "tokens" else None, n if form != "probs" else None)
    tpa.sync_status()


def test_every_outcome_occurs(tpa):
    p, q, x, u, un, n = _inputs(300, 4, 50, 3)
    _, a = _check(tpa, p, x, u, un, q)
    assert set(a.tolist()) == {0, 1, 2, 3, 4}


def test_no_drafts(tpa):
    p, _, x, u, un, _ = _inputs(7, 0, 333, 4)
    _check(tpa, p, x, u, un)
    tpa.sync_status()


def test_borders(tpa):
    """u of 0 and just below 1, weights at the ends of the row and of its parts, rows of zeros, equal rows."""
    V = 1024  # 64 parts of 16
    S = 13
    p = torch.zeros((S, 2, V))
    q = torch.zeros((S, 1, V))
    x = torch.zeros((S, 1), dtype=torch.int32)
    u = torch.full((S, 1), 0.5)
    un = torch.zeros(S)
    q[:, 0, 0] = 1.0                      # drafted token 0, which the target does not have, but for:
    p[0, 0, 1023] = 1.0                   # the last entry alone
    p[1, 0, 8] = 0.5; p[1, 0, 15] = 0.5; un[1] = 0.5            # noqa: E702  a tie: the sum passes u only at 15
    p[2, 0, 7] = 0.5; p[2, 0, 8] = 0.5; un[2] = 1 - 2.0 ** -24  # noqa: E702
    p[3] = 0                              # nothing at all: -1
    p[4, 0] = q[4, 0]; u[4] = 1.0         # noqa: E702  turned down with nothing left: the target's own row
    p[5, 0, 0] = 1.0                      # accepted; the next row is all zeros: -1
    p[6, 0, 0] = 1.0; p[6, 1, 1000] = 1e-30  # noqa: E702
    p[7, 0, 5] = float("nan"); p[7, 0, 9] = 0.25; p[7, 0, 10] = -1.0  # noqa: E702
    p[8, 0] = 1.0 / V; un[8] = 0.5        # noqa: E702
    p[9, 0, 3] = 3e-39; p[9, 0, 700] = 1e-38; un[9] = 0.9     # noqa: E702  subnormal weights
    p[10, 0, 2] = 1.0; p[10, 0, 900] = 2.0 ** -60; un[10] = 1 - 2.0 ** -24  # noqa: E702
    p[11, 0, 0] = 1.0; u[11] = 0.0; p[11, 1, 4] = 1.0         # noqa: E702
    p[12, 0, 15] = 0.5; p[12, 0, 16] = 0.5; un[12] = 0.5      # noqa: E702  a tie between two parts
    t, a = _check(tpa, p, x, u, un, q)
    assert t[12, 0] == 16
    assert t[0, 0] == 1023 and t[1, 0] == 15 and t[2, 0] == 8 and t[3, 0] == -1 and t[4, 0] == 0
    assert t[5].tolist() == [0, -1] and t[6].tolist() == [0, 1000] and t[7, 0] == 9 and t[11].tolist() == [0, 4]
    tpa.sync_status()


def test_small_differences_are_not_lost(tpa):
    """p and q apart by one part in 2^20 to 2^24 of large entries: r is formed exactly."""
    rng = np.random.default_rng(6)
    S, V = 30, 5000
    q = torch.from_numpy(rng.random((S, 1, V), np.float32) + 0.5)
    p = torch.empty((S, 2, V))
    p[:, :1] = q * (1 + torch.from_numpy(rng.integers(-8, 9, (S, 1, V)).astype(np.float32)) * 2.0 ** -23)
    p[:, 1] = 1.0
    x = torch.zeros((S, 1), dtype=torch.int32)
    _check(tpa, p, x, torch.full((S, 1), 2.0), torch.from_numpy(rng.random(S, np.float32)), q)


def test_unnormalised_and_wide_ranges(tpa):
    rng = np.random.default_rng(7)
    S, V = 16, 20011
    p = torch.from_numpy(np.exp(rng.normal(0, 12, (S, 2, V))).astype(np.float32))
    q = torch.from_numpy(np.exp(rng.normal(0, 12, (S, 1, V))).astype(np.float32))
    x = torch.from_numpy(rng.integers(0, V, (S, 1)).astype(np.int32))
    for form in (q, None):
        _check(tpa, p, x, torch.from_numpy(rng.random((S, 1), np.float32)), torch.from_numpy(rng.random(S, np.float32)), form)


def test_bad_tokens_and_counts_are_reported(tpa):
    p, q, x, u, un, n = _inputs(8, 3, 64, 8)
    u[:] = 0
    for bad in (-1, 64, 2 ** 31 - 1, -2 ** 31):
        y = x.clone()
        y[2, 1] = bad
        for form in (q, None):
            _check(tpa, p, y, u, un, form)
            with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
                tpa.sync_status()
            tpa.sync_status()
    n[:] = 3
    n[0], n[1] = -5, 99
    _check(tpa, p, x, u, un, q, n)
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()


def test_strided_sequences_streams_and_graphs(tpa):
    p, q, x, u, un, n = (z.cuda() for z in _inputs(10, 4, 801, 9))
    wide = torch.zeros((10, 7, 801), device="cuda")
    wide[:, 1:6] = p
    want = tpa.verify_drafts(p, x, u, un, q, n)
    got = tpa.verify_drafts(wide[:, 1:6], x, u, un, q, n)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tpa.verify_drafts(p, x, u, un, q, n)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = tpa.verify_drafts(p, x, u, un, q, n)
    u.copy_(torch.rand_like(u))
    un.copy_(torch.rand_like(un))
    want = tpa.verify_drafts(p, x, u, un, q, n)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, kept))
    tpa.sync_status()


def test_rows_past_32_bits(tpa):
    # 3 sequences of 7 rows of 151936, 2^30 entries apart: byte offsets past 2^32
    V, K, S, stride = 151936, 6, 3, 1 << 30
    flat = torch.zeros(2 * stride + (K + 1) * V, device="cuda")
    p, q, x, u, un, n = _inputs(S, K, V, 12)
    far = flat.as_strided((S, K + 1, V), (stride, V, 1))
    far.copy_(p)
    want = oracle_verify(*(z.numpy() for z in (p, x, u, un, q, n)))
    got = tpa.verify_drafts(far, *(z.cuda() for z in (x, u, un, q, n)))
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
