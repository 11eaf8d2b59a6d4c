"""Batches over a paged cache: a sequence's results are its own whatever stands
in the rows beside it, every batch that breaks its description is reported by
the append and by the attention alike, a batch without sequences is no work, and
a captured step goes on while sequences grow.
Sizes on both sides of the borders between kernels."""
import pytest
import torch

from oracle.paged import attend_sequence
from _paged import Batch
from _pipeline import check_guards, guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _rising_keys(b, step):
    """Key dimension 0 rises along each sequence; every query's dimension 0 is 0."""
    b.q[..., 0] = 0
    for s, n in enumerate(b.kv_lens_list):
        j = torch.arange(n)
        page = torch.tensor(b.rows[s])[j // b.page]
        b.k_cache[page.cuda(), :, (j % b.page).cuda(), 0] = (j * step).to(torch.bfloat16).cuda()[:, None]


@pytest.mark.parametrize("q_len,hq,hkv,d", [(1, 4, 1, 128), (1, 32, 8, 128), (3, 4, 2, 64), (5, 16, 4, 128), (2, 12, 1, 64),
                                            (7, 3, 1, 128), (2, 17, 1, 64), (150, 4, 1, 128)])
@pytest.mark.parametrize("window", [0, 20000])
def test_queries_of_other_rows_do_not_matter(tpa, q_len, hq, hkv, d, window):
    """A tile's load brings the rows behind its own: padding, or the next sequence's.  Queries there whose scores rise
    along the keys, or are not numbers, leave every bit of the sequence's own results."""
    lens = [n // hkv for n in (90000, 70000, 80001)]  # some ten steps of 128 keys for every CTA
    b = Batch([q_len] * 3, lens, hq, hkv, d, 16, seed=41, extra=40)
    _rising_keys(b, 1.0)
    n = b.total

    def run():
        return [x.clone() for x in tpa.paged_attn_fwd(*b.cache, b.q, max_q_len=q_len, window=window)]

    b.q[n:] = 0
    want = run()
    for fill in (8.0, -8.0, 3e38, float("inf"), float("-inf"), float("nan")):
        b.q[n:] = 0
        b.q[n:, :, 0] = fill
        assert all(torch.equal(x[:n], y[:n]) for x, y in zip(want, run())), fill
    b.q[n:] = 0
    middle, kept = slice(q_len, 2 * q_len), b.q.clone()
    others = [i for i in range(n) if not q_len <= i < 2 * q_len]
    for fill in (8.0, -8.0, 3e38, float("inf"), float("nan")):
        b.q.copy_(kept)
        b.q[middle, :, 0] = fill
        assert all(torch.equal(x[others], y[others]) for x, y in zip(want, run())), fill
    tpa.sync_status()


# offsets and lengths of three sequences in six rows (and padding behind them), and which sequences they leave as they are
BROKEN = [([0, 5, 2, 6], [20, 3, 33], ()), ([3, 3, 3, 3], [20, 3, 33], ()), ([0, 2, 5, 5000], [20, 3, 33], (0, 1)),
          ([-7, 2, 5, 6], [20, 3, 33], (1, 2)), ([6, 5, 2, 0], [20, 3, 33], ()),
          ([0, 2 ** 31 - 1, -2 ** 31, 6], [20, 3, 33], ()), ([0, 5, 2, 2], [20, 3, 33], ()),
          ([1, 2, 5, 6], [20, 3, 33], (1, 2)), ([0, 5, 5000, 5000], [20, 5000, 33], ()), ([0, 2, 5, 5], [20, 3, -1], (0, 1)),
          ([0, 2, 2, 3], [20, 1000, 33], (0,)), ([0, 2, 2, 3], [20, -2 ** 31, 33], (0,))]


def _broken(off, lens, hq, hkv, extra):
    b = Batch([2, 3, 1], [20, 3, 33], hq, hkv, 64, 16, seed=5, extra=extra)
    b.offsets.copy_(torch.tensor(off, dtype=torch.int32))
    b.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    return b


def _reported(tpa):
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()
    tpa.sync_status()


@pytest.mark.parametrize("off,lens,good", BROKEN)
@pytest.mark.parametrize("max_q", [3, 200])  # the one kernel and the other
def test_broken_batches_are_reported_by_the_attention(tpa, off, lens, good, max_q):
    b = _broken(off, lens, 4, 2, 0)
    bo, o = guarded(b.q.shape, torch.bfloat16)
    bl, lse = guarded(b.q.shape[:2], torch.float32)
    tpa.paged_attn_fwd(*b.cache, b.q, max_q_len=max_q, out=o, lse=lse)
    _reported(tpa)
    check_guards(bo, "o")
    check_guards(bl, "lse")
    for s in good:
        rows = slice(off[s], off[s + 1])
        ref, _, size = attend_sequence(b.q[rows].cpu(), b.sequence(s, b.k_cache), b.sequence(s, b.v_cache))
        # as in test_gpu_paged_attn.py: bf16 probabilities, fp32 scores and sums, a bf16 result
        assert ((o[rows].double().cpu() - ref).abs() <= (2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * ref.abs()).all(), s


@pytest.mark.parametrize("off,lens,good", BROKEN)
@pytest.mark.parametrize("hq,hkv,extra", [(4, 2, 0), (8, 4, 4000)])  # few bytes and many: other kernels
def test_broken_batches_are_reported_by_the_append(tpa, off, lens, good, hq, hkv, extra):
    b = _broken(off, lens, hq, hkv, extra)
    before = b.k_cache.clone(), b.v_cache.clone()
    bq, qo = guarded(b.q.shape, torch.bfloat16)
    tpa.paged_append(*b.cache, b.k, b.v, q=b.q, q_out=qo)
    _reported(tpa)
    check_guards(bq, "q_out")
    # what is written is the value of some row, in a slot that a sequence's own length reaches
    reach = torch.zeros((b.n_pages, b.page), dtype=torch.bool)
    for s, n in enumerate(lens):
        for j in range(max(0, min(n, len(b.rows[s]) * b.page))):
            if b.rows[s][j // b.page] >= 0:
                reach[b.rows[s][j // b.page], j % b.page] = True
    for old, new in zip(before, (b.k_cache, b.v_cache)):
        moved = (old != new).any(-1).any(1).cpu()
        assert not (moved & ~reach).any()
    for s in good:
        pos = torch.arange(lens[s] - (off[s + 1] - off[s]), lens[s])
        page = torch.tensor(b.rows[s])[pos // b.page]
        rows = slice(off[s], off[s + 1])
        assert torch.equal(b.k_cache.cpu()[page, :, pos % b.page], b.k[rows].cpu()), s
        assert torch.equal(b.v_cache.cpu()[page, :, pos % b.page], b.v[rows].cpu()), s
        assert torch.equal(qo[rows], b.q[rows]), s


@pytest.mark.parametrize("extra", [0, 4000])
def test_bad_pages_and_lengths_of_the_append(tpa, extra):
    def run(change, skipped):
        b = Batch([2, 3, 1], [20, 3, 33], 8, 4, 64, 16, seed=5, extra=extra)
        good = b.k_cache.clone(), b.v_cache.clone()
        want = tpa.paged_append(*good, b.pages, b.offsets, b.kv_lens, b.k, b.v, q=b.q)
        page, slot = b.slots()
        change(b)
        got = torch.full_like(b.q, 7.0)
        tpa.paged_append(*b.cache, b.k, b.v, q=b.q, q_out=got)
        _reported(tpa)
        keep = [i for i in range(6) if i not in skipped]
        assert torch.equal(got[keep], want[keep]) and (got[list(skipped)] == 7.0).all() and (got[6:] == 7.0).all()
        for c, w in zip((b.k_cache, b.v_cache), good):
            assert torch.equal(c[page, :, slot][keep], w[page, :, slot][keep])

    for value in (-1, 1000, 2 ** 31 - 1):
        run(lambda b: b.pages[0].__setitem__(1, value), (0, 1))
    for value in (-1, -2 ** 31):
        run(lambda b: b.kv_lens.__setitem__(1, value), (2, 3, 4))
    for value in (49, 2 ** 31 - 1):
        run(lambda b: b.kv_lens.__setitem__(2, value), (5,))


@pytest.mark.parametrize("rows", [70, 2000])
def test_rotation_in_place_and_into_strided_rows(tpa, rows):
    g = torch.Generator().manual_seed(6)
    qkv = torch.randn((rows, 12 * 128), generator=g).to(torch.bfloat16).cuda()
    q, k = qkv[:, :1024].view(rows, 8, 128), qkv[:, 1024:1280].view(rows, 2, 128)
    w = [(1 + 0.3 * torch.randn(128, generator=g)).cuda() for _ in range(2)]
    pos, table = torch.randint(-1, 500, (rows,), generator=g, dtype=torch.int32).cuda(), tpa.rope_table(500, 128)
    want = tpa.qk_norm_rope_fwd(pos, q, k, table, *w)
    fresh = torch.zeros_like(qkv)
    views = fresh[:, :1024].view(rows, 8, 128), fresh[:, 1024:1280].view(rows, 2, 128)
    tpa.qk_norm_rope_fwd(pos, q, k, table, *w, out=views)
    assert all(torch.equal(a, b) for a, b in zip(views, want)) and (fresh[:, 1280:] == 0).all()
    rest = qkv[:, 1280:].clone()
    tpa.qk_norm_rope_fwd(pos, q, k, table, *w, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, 1280:], rest)
    tpa.sync_status()


def test_a_batch_without_sequences(tpa):
    b = Batch([1], [5], 4, 2, 64, 16, seed=1)
    none = dict(pages=b.pages[:0], offsets=b.offsets[:1], kv_lens=b.kv_lens[:0])
    q = tpa.paged_append(b.k_cache, b.v_cache, **none, k=b.k[:0], v=b.v[:0], q=b.q[:0])
    assert q.shape == (0, 4, 64)
    for max_q in (0, 1, 100):
        o, lse = tpa.paged_attn_fwd(b.k_cache, b.v_cache, **none, q=q, max_q_len=max_q)
        assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    tpa.sync_status()


@pytest.mark.parametrize("q_len", [1, 150])
def test_windows_past_32_bits(tpa, q_len):
    b = Batch([q_len], [700], 4, 2, 64, 16, seed=1)
    want = tpa.paged_attn_fwd(*b.cache, b.q, max_q_len=q_len)
    for window in (2 ** 31, 2 ** 32 + 5, 2 ** 63):
        got = tpa.paged_attn_fwd(*b.cache, b.q, max_q_len=q_len, window=window)
        assert all(torch.equal(x, y) for x, y in zip(want, got)), window
    tpa.sync_status()


@pytest.mark.parametrize("drafts", [0, 3, 60])  # a token each, drafts, chunks: every attention kernel
def test_a_captured_sampling_step(tpa, drafts):
    """Append, attention, a projection to the vocabulary and the verification in one graph, replayed while the sequences
    grow over a slice of a wider page table: the same as call by call."""
    S, hq, hkv, d, page, V = 3, 8, 2, 64, 16, 500
    new = drafts + 1
    b = Batch([new] * S, [40 + 4 * new, 7 + 4 * new, 300 + 4 * new], hq, hkv, d, page, seed=4, spare=0, extra=2)
    wide = torch.full((S, b.pages.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + b.pages.shape[1]] = b.pages
    pages = wide[:, 2:2 + b.pages.shape[1]]
    table = tpa.rope_table(600, d)
    g = torch.Generator(device="cuda").manual_seed(2)
    w = [1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    head = torch.randn((hq * d, V), generator=g, device="cuda") * 0.3
    x = torch.randint(0, V, (S, drafts), generator=g, device="cuda", dtype=torch.int32)
    u, un = torch.rand((S, drafts), generator=g, device="cuda"), torch.rand(S, generator=g, device="cuda")

    def step(kc, vc):
        q = tpa.paged_append(kc, vc, pages, b.offsets, b.kv_lens, b.k, b.v, q=b.q, table=table, q_weight=w[0], k_weight=w[1])
        q[S * new:] = 0
        o, lse = tpa.paged_attn_fwd(kc, vc, pages, b.offsets, b.kv_lens, q, max_q_len=new)
        p = torch.softmax(o[:S * new].reshape(S, new, hq * d).float() @ head, -1)
        return (q[:S * new], o[:S * new], lse[:S * new], *tpa.verify_drafts(p, x, u, un))

    eager = b.k_cache.clone(), b.v_cache.clone()
    b.kv_lens -= 3 * new
    lens = b.kv_lens.clone()
    step(eager[0].clone(), eager[1].clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(b.k_cache, b.v_cache)
    for i in range(4):
        for t in (b.q, b.k, b.v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        b.kv_lens.copy_(lens + i * new)
        want = step(*eager)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip((*want, *eager), (*kept, b.k_cache, b.v_cache))), i
    tpa.sync_status()
