"""GPU parity of sampling from logits (tpa_sample_tokens).

Tokens equal the fp64 oracle's: a draw could differ only where u times the kept sum is within 2^-29 of the whole from a
border between two tokens, and a cut where top_p's is; no input here is.  Log-probabilities: the weight
over the sum is off by less than 2^-28 and rounded to fp32 (2^-24), and the logarithm by 2 units in its last place,
2^-22 of itself: 2^-23 + 2^-22 |logp|."""
import math

import numpy as np
import pytest
import torch

from oracle.sample import sample_tokens as oracle_sample
from _pipeline import check_guards, guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _logits(n, v, seed, dtype=torch.float32, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn((n, v), generator=g)
    x.scatter_add_(1, torch.randint(0, v, (n, 12), generator=g), 8 * torch.rand((n, 12), generator=g))
    return x.to(dtype), torch.rand(n, generator=g)


def _column(value, n):
    return value.numpy() if isinstance(value, torch.Tensor) else np.full(n, value)


def _check(tpa, x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, cuda=None):
    n = len(x)
    bt, t = guarded((n,), torch.int32)
    bl, l = guarded((n,), torch.float32)
    dev = lambda z: z.cuda() if isinstance(z, torch.Tensor) else z  # noqa: E731
    tpa.sample_tokens(x.cuda() if cuda is None else cuda, u.cuda(), dev(temperature), dev(top_k), dev(top_p), dev(min_p), out=(t, l))
    check_guards(bt, "tokens")
    check_guards(bl, "logp")
    f32 = lambda z: _column(z, n).astype(np.float32)  # noqa: E731
    want, logp = oracle_sample(x.double().numpy(), u.numpy(), f32(temperature), _column(top_k, n), f32(top_p), f32(min_p))
    got, gl = t.cpu().numpy(), l.double().cpu().numpy()
    assert np.array_equal(got, want), (np.nonzero(got != want), got[got != want], want[got != want])
    some = want >= 0
    assert np.array_equal(np.isnan(gl), ~some)
    assert (np.abs(gl - logp)[some] <= 2.0 ** -23 + 2.0 ** -22 * np.abs(logp[some])).all()
    return got, gl


FORMS = [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=40), dict(top_p=0.9), dict(top_p=0.0), dict(min_p=0.1),
         dict(temperature=0.0), dict(temperature=1.3, top_k=50, top_p=0.8, min_p=0.02), dict(top_k=700, top_p=0.99),
         dict(top_k=300, min_p=1.0), dict(temperature=0.01, top_p=0.5), dict(temperature=50.0, top_p=0.7),
         dict(temperature=30.0, top_k=500)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(1, 1), (3, 2), (4, 7), (5, 65), (3, 999), (2, 4096), (2, 32003)])
@pytest.mark.parametrize("form", FORMS)
def test_against_the_oracle(tpa, n, v, dtype, form):
    x, u = _logits(n, v, n + v, dtype)
    _check(tpa, x, u, **form)
    tpa.sync_status()


@pytest.mark.parametrize("form", [dict(), dict(top_k=50, top_p=0.95), dict(top_p=0.97), dict(top_k=20000)])
def test_full_vocabulary(tpa, form):
    for dtype, v in ((torch.float32, 151936), (torch.bfloat16, 151937)):
        x, u = _logits(3, v, 5, dtype)
        _check(tpa, x, u, **form)
    tpa.sync_status()


def test_every_row_its_own_parameters(tpa):
    n, v = 61, 1501
    x, u = _logits(n, v, 8)
    r = np.random.default_rng(3)
    t = torch.tensor(r.choice([0.0, 0.5, 1.0, 2.0], n), dtype=torch.float32)
    k = torch.tensor(r.choice([-1, 0, 1, 5, 100, 1500, 1501, 9999], n), dtype=torch.int32)
    p = torch.tensor(r.choice([0.0, 0.3, 0.9, 1.0], n), dtype=torch.float32)
    m = torch.tensor(r.choice([0.0, 0.05, 0.5], n), dtype=torch.float32)
    _check(tpa, x, u, t, k, p, m)
    # one kind of parameter as an array, the others numbers
    _check(tpa, x, u, t, 30, 0.9, 0.01)
    _check(tpa, x, u, 0.8, k, 0.9, 0.01)
    tpa.sync_status()


def test_equal_logits_go_by_index(tpa):
    v = 5000
    x = torch.zeros((8, v))
    u = torch.tensor([0.0, 0.5, 1 - 2.0 ** -24, 0.3, 0.3, 0.3, 0.3, 0.3])
    x[4, 17] = 1.0
    x[5, ::2] = -1.0                 # the highest are the odd ones
    x[6] = -0.0
    x[6, 1::2] = 0.0                 # zeros of either sign are one value
    x[7, 100:] = -math.inf
    got, _ = _check(tpa, x, u, top_k=10)
    assert got[:4].tolist() == [0, 5, 9, 3] and got[5:].tolist() == [7, 3, 3]
    _check(tpa, x, u, top_p=0.25)
    _check(tpa, x, u, top_k=4999)
    _check(tpa, x, u, top_k=2600, top_p=0.999)
    _check(tpa, x.to(torch.bfloat16), u, top_k=1000, top_p=0.5)
    tpa.sync_status()


def test_many_equal_values_at_a_cut(tpa):
    """Coarse logits: thousands of tokens of one value at the cut."""
    g = torch.Generator().manual_seed(4)
    x = torch.randint(-3, 3, (6, 40000), generator=g).float()
    u = torch.rand(6, generator=g)
    for form in (dict(top_k=7000), dict(top_p=0.9), dict(top_k=30000, top_p=0.4, temperature=2.0), dict(top_k=1)):
        _check(tpa, x, u, **form)
        _check(tpa, x.to(torch.bfloat16) - 100, u, **form)


def test_masked_and_broken_logits(tpa):
    v = 3001
    x, u = _logits(9, v, 11)
    inf, nan = math.inf, math.nan
    x[0] = -inf
    x[1] = nan
    x[2, 5:] = -inf
    x[3] = -inf
    x[3, v - 1] = -1e30
    x[4, 7] = inf
    x[4, 9] = inf
    x[5, 100:2000] = nan
    x[6] = -3.4e38
    x[6, ::3] = 3.4e38
    x[7, :] = torch.finfo(torch.float32).min
    x[8, 3] = 1e38
    for form in (dict(), dict(top_k=50), dict(top_p=0.9), dict(top_k=3, top_p=0.5, min_p=0.2), dict(temperature=0.0)):
        got, _ = _check(tpa, x, u, **form)
        assert got[0] == -1 and got[1] == -1 and got[2] < 5 and got[3] == v - 1 and got[4] in (7, 9) and got[8] == 3
    tpa.sync_status()  # none of it is an error


@pytest.mark.parametrize("offset", [1000.0, -1000.0, 3e5])
def test_far_from_zero(tpa, offset):
    """The distance from the maximum counts, to all its bits."""
    x, u = _logits(4, 2000, 13)
    x = x + offset
    _check(tpa, x, u, temperature=0.3)
    _check(tpa, x, u, top_k=100, top_p=0.9)


def test_small_logits_of_very_different_sizes(tpa):
    g = torch.Generator().manual_seed(14)
    x = torch.randn((5, 4000), generator=g) * 10.0 ** torch.randint(-30, 1, (5, 4000), generator=g)
    u = torch.rand(5, generator=g)
    for form in (dict(), dict(top_k=1000), dict(top_p=0.6), dict(temperature=1e-3, top_p=0.9), dict(temperature=1e-6)):
        _check(tpa, x, u, **form)


@pytest.mark.parametrize("temperature", [1e-6, 1e-3, 1e3, 1e6])
def test_extreme_temperatures(tpa, temperature):
    x, u = _logits(6, 1700, 15)
    _check(tpa, x, u, temperature=temperature)
    _check(tpa, x, u, temperature=temperature, top_k=30, top_p=0.7)


def test_uniform_numbers_at_their_ends(tpa):
    x, _ = _logits(5, 900, 16)
    x[4] = 0
    for v in (0.0, 1e-30, 0.5, 1 - 2.0 ** -24, 1.0):
        _check(tpa, x, torch.full((5,), v), top_p=0.9)
        _check(tpa, x, torch.full((5,), v))


def test_strides_and_alignments(tpa):
    for dtype in (torch.float32, torch.bfloat16):
        x, u = _logits(7, 517, 17, dtype)
        for skip in range(9):
            wide = torch.full((7, 540), 99.0, dtype=dtype, device="cuda")
            wide[:, skip:skip + 517] = x.cuda()
            _check(tpa, x, u, top_k=20, cuda=wide[:, skip:skip + 517])
            _check(tpa, x, u, cuda=wide[:, skip:skip + 517])


def test_rows_past_32_bits(tpa):
    n, v, stride = 5, 3000, (1 << 30) + 8
    flat = torch.zeros(4 * stride + v, dtype=torch.bfloat16, device="cuda")
    x, u = _logits(n, v, 18, torch.bfloat16)
    far = flat.as_strided((n, v), (stride, 1))
    far.copy_(x)
    _check(tpa, x, u, top_k=30, top_p=0.9, cuda=far)


def test_rows_do_not_depend_on_each_other(tpa):
    x, u = _logits(300, 2048, 19)
    x, u = x.cuda(), u.cuda()
    a = tpa.sample_tokens(x, u, 0.9, 50, 0.9)
    b = tpa.sample_tokens(x[100:107], u[100:107], 0.9, 50, 0.9)
    assert all(torch.equal(i[100:107], j) for i, j in zip(a, b))
    for _ in range(3):
        assert all(torch.equal(i, j) for i, j in zip(a, tpa.sample_tokens(x, u, 0.9, 50, 0.9)))


def test_frequencies(tpa):
    """20000 draws of one distribution: each token's share within five standard deviations."""
    x = torch.tensor([0.0, 1.0, 2.0, -1.0, 0.5]).cuda().expand(20000, 5)
    u = torch.rand(20000, generator=torch.Generator().manual_seed(1)).cuda()
    tokens, logp = tpa.sample_tokens(x.contiguous(), u, 1.0, 4)
    p = torch.softmax(torch.tensor([0.0, 1.0, 2.0, -math.inf, 0.5]), 0)
    share = torch.bincount(tokens.cpu().long(), minlength=5) / 20000
    assert ((share - p).abs() <= 5 * (p * (1 - p) / 20000).sqrt() + 1e-9).all()
    assert ((logp.cpu() - p.log()[tokens.cpu().long()]).abs() < 1e-6).all()


def test_bad_parameters_are_reported(tpa):
    n = 4
    x, u = _logits(n, 100, 20)
    for name, bad in (("temperature", [-1.0, math.nan, 1e-7, math.inf]), ("top_p", [-0.1, 1.5, math.nan, math.inf]),
                      ("min_p", [-0.1, 1.5, math.nan, -math.inf])):
        fine = torch.full((n,), 0.5)
        for i, v in enumerate(bad):
            p = fine.clone()
            p[i] = v
            t, l = tpa.sample_tokens(x.cuda(), u.cuda(), **{name: p.cuda()})
            want = tpa.sample_tokens(x.cuda(), u.cuda(), **{name: fine.cuda()})
            assert t[i] == -1 and torch.isnan(l[i])
            keep = torch.arange(n) != i
            assert torch.equal(t.cpu()[keep], want[0].cpu()[keep])
            with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
                tpa.sync_status()
            tpa.sync_status()


def test_streams_and_graphs(tpa):
    x, u = (z.cuda() for z in _logits(9, 12345, 21))
    want = tpa.sample_tokens(x, u, 0.8, 50, 0.9, 0.01)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tpa.sample_tokens(x, u, 0.8, 50, 0.9, 0.01, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = tpa.sample_tokens(x, u, 0.8, 50, 0.9, 0.01)
    u.copy_(torch.rand_like(u))
    x.copy_(torch.randn_like(x) * 3)
    want = tpa.sample_tokens(x, u, 0.8, 50, 0.9, 0.01)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, kept))
    tpa.sync_status()


def test_no_rows(tpa):
    t, l = tpa.sample_tokens(torch.zeros((0, 10), device="cuda"), torch.zeros(0, device="cuda"))
    assert t.shape == (0,) and l.shape == (0,)


@pytest.mark.parametrize("n,v", [(3, 151936), (70, 20000), (200, 7000)])
@pytest.mark.parametrize("form", [dict(temperature=5.0, top_p=0.97), dict(temperature=1.5, top_p=0.5), dict(temperature=3.0, top_p=0.9, min_p=0.01)])
def test_cuts_among_very_many_tokens(tpa, n, v, form):
    """top_p keeps far more tokens than the ones next to the maximum; every second row has its own, narrow cut."""
    for dtype in (torch.float32, torch.bfloat16):
        x, u = _logits(n, v, 23, dtype)
        t = torch.full((n,), form["temperature"])
        t[1::2] = 0.5
        _check(tpa, x, u, t, 0, form["top_p"], form.get("min_p", 0.0))
    tpa.sync_status()


def test_equal_logits_with_top_p_of_many(tpa):
    x = torch.zeros((5, 30011))
    x[1, ::3] = -2.0
    x[2] = torch.arange(30011) % 7
    x[3, 20000:] = math.inf
    x[4] = -1e38
    u = torch.tensor([0.0, 0.3, 0.6, 0.9, 1 - 2.0 ** -24])
    for p in (0.1, 0.5, 0.999):
        _check(tpa, x, u, top_p=p)
        _check(tpa, x, u, top_k=torch.tensor([0, 29000, 0, 5000, 20], dtype=torch.int32), top_p=p)
    tpa.sync_status()


@pytest.mark.parametrize("offset", [0.0, 300000.0])   # (the second: too far from 0 to be weighed without its maximum)
@pytest.mark.parametrize("kw", [dict(), dict(top_k=900), dict(min_p=1e-25), dict(top_k=torch.full((8,), 990, dtype=torch.int32))])
def test_log_probabilities_next_to_the_cut_off(tpa, offset, kw):
    # u = 0 draws the first token with any weight, here of 2^-14 to 2^-50 of the largest: as whole numbers, down to a few bits
    x = torch.zeros((8, 1000)) + offset
    x[:, 100:] -= 60 if "top_k" in kw else 0
    down = torch.arange(8) * 3.5 + 10
    x[:, 0] = offset - down
    kw = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    t, l = tpa.sample_tokens(x.cuda(), torch.zeros(8, device="cuda"), **kw)
    d = x[:, 0].double() - offset
    whole = (x.double() - offset).exp().sum(1)
    # y of up to 64 as two products and a sum, the sum's logarithm of up to 44: 2^-24 of each, thrice at most
    assert (t == 0).all()
    assert (l.cpu().double() - (d - whole.log())).abs().max() <= 3 * 2.0 ** -24 * (64 + 44)
    tpa.sync_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v,k", [(700, 700, 129), (310, 3000, 700), (301, 9001, 1030), (2, 40000, 3000), (5, 2100, 2049), (301, 2500, 2048)])
def test_top_k_of_many(tpa, n, v, k, dtype):
    # a bound from the threads' maxima, taken apart, and where there are too few of them
    x, u = _logits(n, v, 31, dtype)
    x[1, v // 3:] = -math.inf          # fewer than k are left of a row
    x[0] = (x[0] * 2).round() / 2      # and of another many are equal
    _check(tpa, x, u, 1.0, k, 0.999)
    tpa.sync_status()


@pytest.mark.parametrize("kw", [dict(), dict(top_p=0.9), dict(top_p=0.5, min_p=1e-4), dict(top_k=5000, top_p=0.99), dict(top_k=100000)])
@pytest.mark.parametrize("v", [1 << 24, 3000017])
def test_largest_vocabularies(tpa, v, kw):
    # (against sorted fp64 sums on the device: no border is nearer than they are off, 2^-12 of the whole at the most)
    g = torch.Generator(device="cuda").manual_seed(v)
    x = 2 * torch.randn((2, v), generator=g, device="cuda")
    x[:, 12345] = 24.0                  # half of the weight or so, which u = 0.1 and 0.95 pass by
    x[1] = x[1].flip(0)
    u = torch.tensor([0.95, 0.1], device="cuda")
    t, l = tpa.sample_tokens(x, u, 1.0, **kw)
    for r in range(2):
        w = (x[r].double() - x[r].max()).exp()
        order = torch.sort(x[r], descending=True, stable=True).indices
        k, p, m = kw.get("top_k", v), kw.get("top_p", 1.0), kw.get("min_p", 0.0)
        run = w[order[:k]].cumsum(0)
        n = k if p == 1 else int((run - w[order[:k]] < np.float32(p) * run[-1]).sum())
        kept = torch.zeros_like(w)
        kept[order[:n]] = w[order[:n]]
        kept[kept < np.float32(m)] = 0
        sums = kept.cumsum(0)
        share = sums[int(t[r])] / sums[-1], (sums[int(t[r])] - kept[int(t[r])]) / sums[-1]
        assert kept[int(t[r])] > 0
        assert share[1] - 2.0 ** -12 <= float(u[r]) <= share[0] + 2.0 ** -12
        # the kept sum: as many as top_p keeps to within its own border's distance
        want = (w[int(t[r])] / sums[-1]).log()
        assert abs(float(l[r]) - float(want)) <= 2.0 ** -11 + 2.0 ** -22 * abs(float(want))
    tpa.sync_status()
