"""GPU parity of the paged attention (tpa_paged_attn_fwd) against fp64.

Tolerances.  A probability enters the second product as bf16: off by 2^-8 of
itself.  What is fp32 (scores: 16 or fewer additions of the matrix unit, each
within 2^-23 of the partial sums, 8 at most in these inputs; exponentials 2^-22;
sums of at most 512 terms a lane) changes a probability by less than 2^-14.  So O
is within (2^-8 + 2^-14) sum p |v|, and half a step of its own, 2^-8 |O|; LSE is
within 2^-14 plus its own rounding."""

import numpy as np
import pytest
import torch

from oracle.paged import attend_sequence
from synth import random_small_sequences
from _paged import Batch
from _pipeline import check_guards, guarded, pack_and_upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _check_values(b, o, lse, window=0, scale=None, only=None):
    at = 0
    for s, n in enumerate(b.q_lens):
        rows = slice(at, at + n)
        at += n
        if n == 0 or (only is not None and s not in only):
            continue
        k, v = b.sequence(s, b.k_cache), b.sequence(s, b.v_cache)
        ref, rl, size = attend_sequence(b.q[rows].cpu(), k, v, window, scale)
        got, gl = o[rows].double().cpu(), lse[rows].double().cpu()
        assert torch.isfinite(got).all(), f"sequence {s}"
        off = (got - ref).abs() - ((2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * ref.abs())
        assert off.max() <= 0, f"sequence {s}: {off.max():.3e} past the bound"
        none = torch.isinf(rl)
        assert torch.equal(torch.isinf(gl) & (gl < 0), none), f"sequence {s}: rows that see nothing"
        assert (got[none] == 0).all()
        fine = ~none
        assert ((gl[fine] - rl[fine]).abs() <= 2.0 ** -14 + 2.0 ** -23 * rl[fine].abs()).all(), f"sequence {s}: LSE"


def _run(tpa, b, window=0, scale=None, max_q=None):
    bo, o = guarded(b.q.shape, torch.bfloat16)
    bl, lse = guarded(b.q.shape[:2], torch.float32)
    o.fill_(7.0)
    lse.fill_(7.0)
    q_max = max(max(b.q_lens, default=1), 1) if max_q is None else max_q
    hq, hkv = b.hq, b.hkv
    nbytes = tpa.paged_attn_workspace_bytes(q_max, hq, hkv, b.d)
    bw, ws = guarded((nbytes // 4 + 4096,), torch.int32)
    ws = ws.view(torch.uint8)
    skip = -ws.data_ptr() % 256
    tpa.paged_attn_fwd(*b.cache, b.q, max_q_len=q_max, window=window, softmax_scale=scale, out=o, lse=lse,
                       workspace=ws[skip:skip + nbytes])
    for buf, what in ((bo, "o"), (bl, "lse"), (bw, "workspace")):
        check_guards(buf, what)
    assert (o[b.total:] == 7.0).all() and (lse[b.total:] == 7.0).all()
    return o, lse


CASES = [  # q_lens, kv_lens, hq, hkv, d, page, extra rows
    ([1], [1], 1, 1, 64, 16, 0), ([1], [1], 8, 1, 128, 16, 1), ([1] * 5, [127, 128, 129, 1, 256], 4, 2, 128, 32, 2),
    ([1] * 9, [1, 16, 17, 1033, 5, 400, 64, 65, 2], 32, 8, 128, 16, 3), ([1] * 3, [700, 3000, 15], 16, 1, 128, 64, 0),
    ([1] * 4, [300, 31, 33, 2000], 32, 1, 64, 128, 0), ([1, 1], [5000, 77], 17, 1, 128, 16, 0),
    ([5, 0, 1, 3, 0], [5, 40, 129, 300, 0], 8, 2, 128, 64, 10), ([2, 4, 8], [2, 1200, 9], 6, 2, 64, 16, 0),
    ([9, 9], [2000, 9], 5, 5, 128, 32, 0), ([33], [33], 4, 4, 64, 16, 3), ([200], [200], 8, 2, 128, 16, 0),
    ([130, 1, 257, 7], [700, 80, 257, 1500], 8, 2, 128, 64, 5), ([100], [1000], 3, 1, 64, 128, 0),
    ([129, 64], [129, 999], 7, 1, 128, 32, 0), ([0, 0], [0, 30], 4, 2, 64, 16, 3), ([300], [4000], 24, 8, 128, 128, 0),
    ([65], [640], 10, 2, 64, 32, 0), ([40, 40], [41, 1000], 32, 1, 128, 16, 0),
    ([1, 1, 3], [900, 64, 130], 64, 1, 128, 16, 1), ([1, 2], [333, 3], 66, 2, 64, 32, 0)]


@pytest.mark.parametrize("window", [0, 1, 100, 300])
@pytest.mark.parametrize("case", CASES)
def test_against_the_oracle(tpa, case, window):
    b = Batch(*case[:6], seed=23, extra=case[6])
    o, lse = _run(tpa, b, window)
    tpa.sync_status()
    _check_values(b, o, lse, window)


@pytest.mark.parametrize("case", [([7], [3], 8, 2, 128, 16, 2), ([200, 5], [60, 0], 4, 2, 64, 32, 0),
                                  ([1, 1], [0, 9], 4, 1, 128, 16, 0), ([300], [170], 16, 2, 128, 64, 0)])
def test_rows_that_see_nothing(tpa, case):
    b = Batch(*case[:6], seed=29, extra=case[6])
    o, lse = _run(tpa, b)
    tpa.sync_status()
    _check_values(b, o, lse)


def test_scale_and_large_scores(tpa):
    b = Batch([1, 3, 150], [500, 900, 300], 8, 2, 128, 16, seed=3)
    for scale in (0.5, 0.01):
        o, lse = _run(tpa, b, scale=scale)
        # scores up to 0.5 x 60: their fp32 error grows with them, by 0.5 / 0.088 of what the bound counts
        b_ok = 1 if scale < 0.1 else 8
        at = 0
        for s, n in enumerate(b.q_lens):
            ref, rl, size = attend_sequence(b.q[at:at + n].cpu(), b.sequence(s, b.k_cache), b.sequence(s, b.v_cache), 0, scale)
            off = (o[at:at + n].double().cpu() - ref).abs() - ((2.0 ** -8 + b_ok * 2.0 ** -14) * size + 2.0 ** -8 * ref.abs())
            assert off.max() <= 0
            assert ((lse[at:at + n].double().cpu() - rl).abs() <= b_ok * 2.0 ** -14 + 2.0 ** -23 * rl.abs()).all()
            at += n


@pytest.mark.parametrize("q_len", [1, 6, 140])
def test_growing_scores(tpa, q_len):
    """Every key's score is above the ones before it: the running maximum moves all the time."""
    b = Batch([q_len], [1500], 4, 1, 128, 16, seed=5)
    b.q[:] = 0
    b.q[..., 0] = 1.0
    j = torch.arange(1500)
    page = torch.tensor(b.rows[0])[j // 16]
    b.k_cache[page.cuda(), 0, (j % 16).cuda(), 0] = (j.float() * 1.5).to(torch.bfloat16).cuda()
    o, lse = _run(tpa, b)
    _check_values(b, o, lse)


@pytest.mark.parametrize("q_len,group", [(1, 4), (4, 4), (150, 4), (600, 2)])
@pytest.mark.parametrize("window", [0, 200])
def test_slots_that_nobody_sees_may_hold_anything(tpa, q_len, group, window):
    kv = 1003
    b = Batch([q_len, q_len], [kv, kv - 1], group, 1, 128, 64, seed=7)
    clean = [x.clone() for x in _run(tpa, b, window)]
    for s, n in enumerate(b.kv_lens_list):
        last = b.rows[s][n // 64]
        b.k_cache[last, :, n % 64:] = float("nan")
        b.v_cache[last, :, n % 64:] = float("nan") if s else float("inf")
        first = n - q_len - window + 1 if window else 0
        if first > 0:
            page = b.rows[s][first // 64]
            b.k_cache[page, :, :first % 64] = float("inf")
            b.v_cache[page, :, :first % 64] = float("nan")
            b.pages[s, :first // 64] = -1  # recycled
    spare = [i for i in range(b.n_pages) if not any(i in r for r in b.rows)]
    b.k_cache[spare] = float("nan")
    b.v_cache[spare] = float("nan")
    dirty = _run(tpa, b, window)
    tpa.sync_status()
    assert all(torch.equal(x, y) for x, y in zip(clean, dirty))


@pytest.mark.parametrize("q_len", [1, 3, 200])
def test_shared_pages(tpa, q_len):
    b = Batch([q_len] * 6, [640 + q_len + i for i in range(6)], 8, 2, 128, 64, seed=9)
    for s in range(1, 6):  # the first ten pages of each group of three are the first's
        g = s - s % 3
        b.rows[s][:10] = b.rows[g][:10]
        b.pages[s, :10] = b.pages[g, :10]
    o, lse = _run(tpa, b)
    _check_values(b, o, lse)


@pytest.mark.parametrize("n", [257, 1000, 2500])
def test_many_sequences(tpa, n):
    rng = np.random.default_rng(n)
    b = Batch([int(x) for x in rng.integers(0, 3, n)], [int(x) for x in rng.integers(2, 90, n)], 4, 2, 64, 16, seed=n)
    o, lse = _run(tpa, b)
    tpa.sync_status()
    _check_values(b, o, lse, only=set(range(0, n, 37)) | {n - 1})


@pytest.mark.parametrize("case", [(64, 1, 300, 3000, 32, 8, 128), (16, 5, 1000, 8000, 32, 8, 128),
                                  (16, 8, 1000, 8000, 16, 4, 64), (12, 1, 990, 1030, 32, 8, 128),
                                  (24, (1, 32, 33, 70, 140), 300, 2500, 8, 2, 128), (24, (1, 10, 70), 300, 2500, 16, 2, 64)])
def test_tiles_that_follow_one_another(tpa, case):
    """Many steps and several tiles for every CTA: a tile's last, ragged step runs beside the loads of those before it."""
    n, q_len, least, most, hq, hkv, d = case
    rng = np.random.default_rng(17)
    q_lens = [q_len] * n if isinstance(q_len, int) else [int(x) for x in rng.choice(q_len, n)]
    b = Batch(q_lens, [int(x) for x in rng.integers(least, most, n)], hq, hkv, d, 16, seed=17)
    first = [x.clone() for x in _run(tpa, b)]
    _check_values(b, *first)
    for _ in range(6):
        assert all(torch.equal(x, y) for x, y in zip(first, _run(tpa, b)))
    tpa.sync_status()


@pytest.mark.parametrize("q_lens", [(1, 3, 2), (200, 7, 64)])
def test_windows_past_every_position(tpa, q_lens):
    b = Batch(list(q_lens), [700, 5, 129], 8, 2, 128, 16, seed=21)  # the second has more new tokens than cached ones, or few
    want = _run(tpa, b)
    for window in (701, 1 << 30, (1 << 30) + 1, 2 ** 31 - 1):
        assert all(torch.equal(x, y) for x, y in zip(want, _run(tpa, b, window)))
    tpa.sync_status()
    _check_values(b, *want)


@pytest.mark.parametrize("q_len", [1, 5])
def test_one_long_sequence(tpa, q_len):
    b = Batch([q_len], [70001], 8, 2, 128, 128, seed=4)
    o, lse = _run(tpa, b)
    tpa.sync_status()
    _check_values(b, o, lse)


def test_longer_chunks_than_said(tpa):
    b = Batch([1, 90, 4], [300, 500, 4], 8, 2, 128, 16, seed=6)
    o, lse = _run(tpa, b, max_q=1)
    _check_values(b, o, lse)
    o, lse = _run(tpa, b, max_q=5000)
    _check_values(b, o, lse)


def test_shorter_chunks_than_said(tpa):
    b = Batch([1, 0, 2, 1], [300, 500, 2, 4000], 8, 2, 128, 16, seed=6, extra=2)
    o, lse = _run(tpa, b, max_q=64)
    _check_values(b, o, lse)


def test_query_slices(tpa):
    b = Batch([3, 140], [10, 300], 4, 2, 128, 16, seed=2)
    want = _run(tpa, b)
    qkv = torch.randn((143, 8 * 128), device="cuda").to(torch.bfloat16)
    qkv[:, :512] = b.q.view(143, 512)
    got = tpa.paged_attn_fwd(*b.cache, qkv[:, :512].view(143, 4, 128), max_q_len=140)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_bad_batches_are_reported(tpa):
    def run(change, hurt, q=(1, 3, 150)):
        b = Batch(list(q), [400, 300, 500], 8, 2, 128, 16, seed=8)
        change(b)
        o, lse = _run(tpa, b)
        with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
            tpa.sync_status()
        tpa.sync_status()
        _check_values(b, o, lse, only={0, 1, 2} - hurt)
        return o, lse

    for q in ((1, 3, 150), (1, 1, 2)):
        for value in (-1, 2 ** 31 - 1, 10 ** 6):
            run(lambda b: b.pages[0].__setitem__(3, value), {0}, q)
        for value in (-1, 2 ** 31 - 1, 501 + 16):
            o, lse = run(lambda b: b.kv_lens.__setitem__(2, value), {2}, q)
            assert (o[q[0] + q[1]:] == 7.0).all() and (lse[q[0] + q[1]:] == 7.0).all()


@pytest.mark.parametrize("q_lens", [(2, 3, 1), (200, 3, 1)])
def test_unordered_offsets_end_and_stay_inside(tpa, q_lens):
    n = sum(q_lens)
    for off in ([0, 5, 2, n], [3, 3, 3, 3], [0, 2, 5, 1000], [-7, 2, 5, n], [n, 5, 2, 0], [0, 2 ** 31 - 1, -2 ** 31, n]):
        b = Batch(list(q_lens), [220, 3, 33], 4, 2, 64, 16, seed=5)
        b.offsets.copy_(torch.tensor(off, dtype=torch.int32))
        b.total = n
        _run(tpa, b)
        try:
            tpa.sync_status()
        except tpa.TpaError as e:
            assert e.name == "TPA_ERR_INVALID_ARG"


@pytest.mark.parametrize("q_len", [2, 130])
def test_a_cache_past_32_bits(tpa, q_len):
    n_pages, hkv, page, d = 20480, 8, 128, 128
    b = Batch([q_len, q_len], [150, q_len], 8, hkv, d, page, seed=3)
    kc = torch.zeros((n_pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros((n_pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    want = _run(tpa, b)
    far = {p: n_pages - 1 - 1000 * i for i, p in enumerate(sorted(set(sum(b.rows, [])) - {-1}))}
    for p, f in far.items():
        kc[f], vc[f] = b.k_cache[p], b.v_cache[p]
    b.k_cache, b.v_cache = kc, vc
    b.rows = [[far.get(p, -1) for p in r] for r in b.rows]
    b.pages.copy_(torch.tensor(b.rows, dtype=torch.int32))
    got = _run(tpa, b)
    tpa.sync_status()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("q_len,kv", [(1, 3001), (4, 3001), (150, 3001)])
def test_streams_graphs_and_repeats(tpa, q_len, kv):
    b = Batch([q_len, q_len], [kv, kv // 3], 8, 2, 128, 16, seed=4)
    want = [x.clone() for x in _run(tpa, b)]
    again = _run(tpa, b)
    assert all(torch.equal(x, y) for x, y in zip(want, again))
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for st in side:  # two calls at once
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(tpa.paged_attn_fwd(*b.cache, b.q, max_q_len=q_len))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g in got for x, y in zip(want, g))
    graphs, kept = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            kept.append(tpa.paged_attn_fwd(*b.cache, b.q, max_q_len=q_len))
    # other lengths, read by the kernels when the graphs run
    b.kv_lens.copy_(torch.tensor([kv // 2, kv // 3 - 5], dtype=torch.int32))
    b.kv_lens_list = [kv // 2, kv // 3 - 5]
    want = _run(tpa, b)
    for st, g in zip(side, graphs):
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for k in kept for x, y in zip(want, k))
    _check_values(b, *want)
    tpa.sync_status()


@pytest.mark.parametrize("raw", [False, True])
def test_results_of_a_call_on_another_stream_are_its_own(tpa, raw):
    """What the current stream still writes to memory that was given back does not reach the outputs of a call on
    another one, nor the other way round its workspace memory that is handed out again."""
    b = Batch([2] * 8, [3000] * 8, 8, 2, 128, 16, seed=14)
    table = tpa.rope_table(3000, 128)
    p, x = torch.softmax(torch.randn((4, 3, 9000), device="cuda"), -1), torch.randint(0, 9000, (4, 2), device="cuda").int()
    u, un = torch.rand((4, 2), device="cuda"), torch.rand(4, device="cuda")
    at = torch.arange(b.total, device="cuda", dtype=torch.int32)

    def calls(stream=None):
        q, k = tpa.qk_norm_rope_fwd(at, b.q, b.k, table, stream=stream)
        return (tpa.rope_table(3000, 128, stream=stream), q, k, *tpa.qk_norm_rope_bwd(at, b.q, b.k, None, None, table, stream=stream)[:2],
                tpa.paged_append(*b.cache, b.k, b.v, q=b.q, table=table, stream=stream),
                *tpa.paged_attn_fwd(*b.cache, b.q, max_q_len=2, stream=stream), *tpa.verify_drafts(p, x, u, un, stream=stream))

    want = [z.clone() for z in calls()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    mine = [torch.empty_like(z) for z in want for _ in range(3)]
    torch.cuda._sleep(100_000_000)
    for z in mine:
        z.fill_(7)
    del mine, z
    got = calls(side.cuda_stream if raw else side)
    after = [torch.empty_like(z).fill_(7) for z in want]  # noqa: F841
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    tpa.sync_status()


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 8, 1)])
def test_the_sampled_policy_is_the_trained_one(tpa, d, hq, hkv):
    """A packed tree's attention on the training side, and the same sequences on the sampling side: their prompts in
    chunks, then token by token, over pages that share what the tree shares.  Both are held to the oracle's causal
    attention by their own bounds, so their difference by the sum."""
    rng = np.random.default_rng(31)
    seqs = random_small_sequences(rng, 5, 120, 3, min_len=20)
    T, page = 256, 16
    tree, dtree, mask = pack_and_upload(tpa, seqs, T)
    arr = tree.arrays()
    g = torch.Generator().manual_seed(1)
    B = tree.n_trees
    qkv = torch.randn((B, T, (hq + 2 * hkv) * d), generator=g).to(torch.bfloat16).cuda()
    q, k = qkv[..., :hq * d].view(B, T, hq, d), qkv[..., hq * d:(hq + hkv) * d].view(B, T, hkv, d)
    v = qkv[..., (hq + hkv) * d:].reshape(B, T, hkv, d).contiguous()
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    table = tpa.rope_table(T, d)
    qr, kr = tpa.qk_norm_rope_fwd(dtree, q, k, table, wq, wk)
    o_tree, _ = tpa.tree_attn_fwd(dtree, mask, qr, kr, v)

    lens = [len(s) for s in seqs]
    width = -(-max(lens) // page)
    kc = torch.full((len(seqs) * width, hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    pages = torch.randperm(len(seqs) * width, generator=g).to(torch.int32).view(len(seqs), width).cuda()
    rows = [torch.from_numpy(arr["seq_pos"][a:b].astype(np.int64)) + int(arr["seq_tree"][s]) * T
            for s, (a, b) in enumerate(zip(arr["seq_off"][:-1], arr["seq_off"][1:]))]
    flat = [x.reshape(B * T, *x.shape[2:]) for x in (q, k, v)]
    got = [[] for _ in seqs]
    done = [0] * len(seqs)
    plan = [[min(n - 6, 13) for n in lens], [n - 6 - min(n - 6, 13) for n in lens], [4] * len(seqs), [1] * len(seqs), [1] * len(seqs)]
    for news in plan:
        at = torch.cat([rows[s][done[s]:done[s] + n] for s, n in enumerate(news)]).cuda()
        offsets = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
        done = [a + n for a, n in zip(done, news)]
        kv_lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        qn, kn, vn = (x[at] for x in flat)
        y = tpa.paged_append(kc, vc, pages, offsets, kv_lens, kn, vn, q=qn, table=table, q_weight=wq, k_weight=wk)
        assert torch.equal(y, qr.reshape(B * T, hq, d)[at])  # the same rows, rotated alike
        o, _ = tpa.paged_attn_fwd(kc, vc, pages, offsets, kv_lens, y, max_q_len=max(news))
        for s in range(len(seqs)):
            got[s].append(o[int(offsets[s]):int(offsets[s + 1])])
    tpa.sync_status()
    for s, n in enumerate(lens):
        want = o_tree.reshape(B * T, hq, d)[rows[s].cuda()].double().cpu()
        x = torch.cat(got[s]).double().cpu()
        kk, vv = (z.reshape(B * T, hkv, d)[rows[s].cuda()].cpu() for z in (kr, v))
        ref, _, size = attend_sequence(qr.reshape(B * T, hq, d)[rows[s].cuda()].cpu(), kk, vv)
        bound = (2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * ref.abs()
        assert ((x - ref).abs() <= bound).all()
        assert ((x - want).abs() <= 2 * bound).all()


def test_sampling_step_with_drafts(tpa):
    """Drafted tokens through append, attention, a projection to the vocabulary and the verification."""
    from oracle.verify import verify_drafts as oracle_verify
    S, K, V = 5, 3, 1000
    b = Batch([K + 1] * S, [50, 4, 300, 129, 17], 8, 2, 64, 16, seed=12)
    table = tpa.rope_table(400, 64)
    q = tpa.paged_append(*b.cache, b.k, b.v, q=b.q, table=table)
    o, lse = tpa.paged_attn_fwd(*b.cache, q, max_q_len=K + 1)
    b.q = q
    _check_values(b, o, lse)
    head = torch.randn((8 * 64, V), device="cuda") * 0.3
    p = torch.softmax(o.reshape(S, K + 1, 8 * 64).float() @ head, -1)
    d = torch.softmax(torch.log(p[:, :K]) + 0.3 * torch.randn((S, K, V), device="cuda"), -1)
    x = torch.multinomial(d.reshape(S * K, V), 1).view(S, K).to(torch.int32)
    u, un = torch.rand((S, K), device="cuda"), torch.rand(S, device="cuda")
    tokens, n = tpa.verify_drafts(p, x, u, un, draft_probs=d)
    tpa.sync_status()
    want = oracle_verify(*(z.cpu().numpy() for z in (p, x, u, un, d)))
    assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(n.cpu().numpy(), want[1])
