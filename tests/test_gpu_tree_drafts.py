"""GPU parity of the drafted trees' operators: masks and positions, attention
under masks, accepted paths, and the cache with a path's keys and values moved.

Whole numbers and moved values are equal to the oracle's.  Attention has the
bounds of the paged attention without a tree (probabilities bf16 operands of the
second product, 2^-8 of sum p |v|; what is fp32, 2^-14 of it; O rounded once, 2^-8 |O|;
LSE 2^-14 and its rounding)."""
import numpy as np
import pytest
import torch

from oracle.draft import accept, attend_tree, masks as oracle_masks
from _paged import Batch
from _pipeline import check_guards, guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _trees(q_lens, seed, form="wide"):
    r = np.random.default_rng(seed)
    trees = []
    for n in q_lens:
        if form == "chain":
            t = list(range(-1, n - 1))
        elif form == "star":
            t = [-1] + [0] * (n - 1)
        elif form == "loose":  # several roots, any earlier parent
            t = [int(r.integers(-1, i)) if i else -1 for i in range(n)]
        else:
            t = [-1] + [int(r.integers((i - 1) // 4, (i - 1) // 2 + 1)) for i in range(1, n)]
        trees.append(t[:n])
    return trees


def _flat(trees):
    return _i32([p for t in trees for p in t])


@pytest.mark.parametrize("form", ["wide", "chain", "star", "loose"])
@pytest.mark.parametrize("q_lens,kv_lens,extra", [([1], [1], 0), ([5, 0, 33], [5, 0, 900], 3), ([64, 32, 31, 65], [64, 100, 31, 70], 0),
                                                  ([1024, 1], [2000, 1], 5), ([7, 200], [3, 100], 1)])
@pytest.mark.parametrize("window", [0, 1, 3])
def test_masks(tpa, q_lens, kv_lens, extra, form, window):
    trees = _trees(q_lens, 3, form)
    n, most = sum(q_lens), max(q_lens)
    words = -(-most // 32)
    parents = torch.cat([_flat(trees), _i32([-7] * extra)]).cuda()
    offsets, lens = _i32([0] + list(np.cumsum(q_lens))).cuda(), _i32(kv_lens).cuda()
    bp, p = guarded((n + extra,), torch.int32)
    bm, m = guarded((n + extra, words), torch.int32)
    p.fill_(77)
    m.fill_(77)
    tpa.draft_masks(parents, offsets, lens, most, window, out=(p, m))
    check_guards(bp, "positions")
    check_guards(bm, "masks")
    want = [oracle_masks(t, b - len(t), words, window) for t, b in zip(trees, kv_lens)]
    assert p[:n].tolist() == [x for w in want for x in w[0]]
    assert m[:n].tolist() == [x for w in want for x in w[1]]
    assert (p[n:] == 77).all() and (m[n:] == 77).all()
    tpa.sync_status()


def test_broken_parents_are_reported(tpa):
    offsets, lens = _i32([0, 4, 8]).cuda(), _i32([10, 20]).cuda()
    for at, bad in ((1, 1), (2, 3), (5, -2), (0, 0), (3, 2 ** 31 - 1), (7, -2 ** 31)):
        parents = _i32([-1, 0, 0, 1, -1, 0, 1, 2])
        parents[at] = bad
        p, m = tpa.draft_masks(parents.cuda(), offsets, lens, 4)
        fixed = parents.tolist()
        fixed[at] = -1
        want = [oracle_masks(fixed[i:i + 4], b, 1) for i, b in ((0, 6), (4, 16))]
        assert p.tolist() == [x for w in want for x in w[0]] and m.tolist() == [x for w in want for x in w[1]]
        with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
            tpa.sync_status()
        x = torch.zeros(8, dtype=torch.int32, device="cuda")  # every token fits
        tokens, path, n = tpa.accept_drafts(parents.cuda(), offsets, x, x, 4)
        with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
            tpa.sync_status()
        assert at not in path[at // 4].tolist()[1:] or at % 4 == 0


def test_broken_offsets_are_reported(tpa):
    parents, lens = _i32([-1, 0, 0, 1]).cuda(), _i32([10, 20]).cuda()
    x = torch.zeros(4, dtype=torch.int32, device="cuda")
    for off in ([0, 2, 5], [0, 3, 2], [1, 2, 4], [-1, 2, 4]):
        for call in (lambda o: tpa.draft_masks(parents, o, lens, 4), lambda o: tpa.accept_drafts(parents, o, x, x, 3)):
            call(_i32(off).cuda())
            with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
                tpa.sync_status()
    # more new tokens than the masks have bits for
    many = torch.full((40,), -1, dtype=torch.int32, device="cuda")
    _, m = tpa.draft_masks(many, _i32([0, 40]).cuda(), _i32([40]).cuda(), 32)
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()


# ------------------------------------------------------------------ attention

def _seen(trees, kv_lens, window=0):
    """[n, kv] of each sequence, by walking up from each token."""
    out = []
    for t, b in zip(trees, kv_lens):
        n = len(t)
        seen = torch.zeros((n, b), dtype=torch.bool)
        for i in range(n):
            up, depth = i, 0
            while up >= 0:
                if (not window or depth < window) and b - n + up >= 0:
                    seen[i, b - n + up] = True
                up, depth = t[up], depth + 1
            low = max(0, b - n + depth - 1 - window + 1) if window else 0
            seen[i, low:max(b - n, 0)] = True
        out.append(seen)
    return out


def _check_attention(b, o, lse, seen):
    at = 0
    for s, n in enumerate(b.q_lens):
        rows = slice(at, at + n)
        at += n
        if n == 0:
            continue
        ref, rl, size = attend_tree(b.q[rows].cpu(), b.sequence(s, b.k_cache), b.sequence(s, b.v_cache), seen[s])
        got, gl = o[rows].double().cpu(), lse[rows].double().cpu()
        assert torch.isfinite(got).all()
        off = (got - ref).abs() - ((2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * ref.abs())
        assert off.max() <= 0, f"sequence {s}: {off.max():.3e} past the bound"
        none = torch.isinf(rl)
        assert torch.equal(torch.isinf(gl) & (gl < 0), none) and (got[none] == 0).all()
        assert ((gl[~none] - rl[~none]).abs() <= 2.0 ** -14 + 2.0 ** -23 * rl[~none].abs()).all(), f"sequence {s}: LSE"


def _attend(tpa, b, positions, masks, window=0, max_q=None):
    bo, o = guarded(b.q.shape, torch.bfloat16)
    bl, lse = guarded(b.q.shape[:2], torch.float32)
    o.fill_(7.0)
    lse.fill_(7.0)
    tpa.paged_attn_tree_fwd(*b.cache, b.q, masks, max_q_len=max_q or max(max(b.q_lens), 1), positions=positions, window=window,
                            out=o, lse=lse)
    check_guards(bo, "o")
    check_guards(bl, "lse")
    assert (o[b.total:] == 7.0).all() and (lse[b.total:] == 7.0).all()
    return o, lse


CASES = [  # q_lens, kv_lens, hq, hkv, d, page, extra rows
    ([1], [1], 1, 1, 64, 16, 0), ([1, 1], [300, 5], 8, 1, 128, 16, 1), ([4, 4, 3], [4, 500, 131], 4, 1, 128, 32, 2),
    ([8] * 5, [300, 8, 130, 128, 1000], 32, 8, 128, 16, 0), ([8, 0, 5, 1], [700, 0, 133, 257], 8, 2, 64, 64, 3),
    ([16, 9], [900, 9], 2, 2, 64, 128, 0), ([1, 2], [333, 3], 64, 2, 64, 32, 0), ([32], [32], 1, 1, 128, 16, 0),
    ([33], [400], 4, 4, 128, 16, 0), ([64, 20, 1, 47], [64, 1000, 129, 700], 32, 8, 128, 32, 4),
    ([100, 3], [229, 500], 8, 2, 64, 16, 0), ([200], [200], 10, 2, 128, 128, 0), ([300, 129], [4000, 130], 6, 2, 64, 64, 1),
    ([1024], [1500], 2, 1, 128, 64, 0), ([40], [1000], 66, 2, 128, 16, 0), ([37], [5000], 5, 1, 128, 128, 0)]


@pytest.mark.parametrize("form,window", [("wide", 0), ("wide", 3), ("wide", 150), ("loose", 0), ("star", 40), ("chain", 0)])
@pytest.mark.parametrize("case", CASES)
def test_attention(tpa, case, form, window):
    b = Batch(*case[:6], seed=31, extra=case[6])
    trees = _trees(b.q_lens, 5, form)
    parents = torch.cat([_flat(trees), _i32([0] * case[6])]).cuda()
    positions, masks = tpa.draft_masks(parents, b.offsets, b.kv_lens, max(b.q_lens), window)
    masks[b.total:] = 0
    o, lse = _attend(tpa, b, positions, masks, window)
    tpa.sync_status()
    _check_attention(b, o, lse, _seen(trees, b.kv_lens_list, window))


@pytest.mark.parametrize("case", CASES)
def test_chains_are_the_attention_without_a_tree(tpa, case):
    b = Batch(*case[:6], seed=33, extra=case[6])
    most = max(b.q_lens)
    parents = torch.cat([_flat(_trees(b.q_lens, 0, "chain")), _i32([0] * case[6])]).cuda()
    positions, masks = tpa.draft_masks(parents, b.offsets, b.kv_lens, most)
    o, lse = tpa.paged_attn_tree_fwd(*b.cache, b.q, masks, most, positions=positions)
    want = tpa.paged_attn_fwd(*b.cache, b.q, most)
    n = b.total
    assert torch.equal(o[:n], want[0][:n]) and torch.equal(lse[:n], want[1][:n])


@pytest.mark.parametrize("q_lens,kv_lens", [([5], [3]), ([40], [10]), ([3, 70], [0, 60])])
def test_more_new_tokens_than_cached_ones(tpa, q_lens, kv_lens):
    """base < 0: the first tokens have no slot."""
    b = Batch(q_lens, kv_lens, 4, 2, 64, 16, seed=35)
    trees = _trees(q_lens, 7)
    positions, masks = tpa.draft_masks(_flat(trees).cuda(), b.offsets, b.kv_lens, max(q_lens))
    o, lse = _attend(tpa, b, positions, masks)
    tpa.sync_status()
    _check_attention(b, o, lse, _seen(trees, kv_lens))


@pytest.mark.parametrize("n,kv", [(6, 200), (80, 333)])
def test_any_bits(tpa, n, kv):
    """Masks that are no tree's: bits of later tokens do not count, and a token may see nothing of the new ones."""
    b = Batch([n, n], [kv, n], 8, 2, 128, 16, seed=36)
    words = -(-n // 32)
    g = torch.Generator().manual_seed(2)
    masks = torch.randint(-2 ** 31, 2 ** 31, (2 * n, words), generator=g, dtype=torch.int64).to(torch.int32)
    masks[3] = 0
    masks[n + 2] = 0  # and nothing is cached before: the row sees nothing
    seen = []
    for s, k in enumerate((kv, n)):
        m = torch.zeros((n, k), dtype=torch.bool)
        m[:, :k - n] = True
        for i in range(n):
            for j in range(i + 1):
                m[i, k - n + j] = bool(int(masks[s * n + i, j // 32]) >> j % 32 & 1)
        seen.append(m)
    o, lse = _attend(tpa, b, None, masks.cuda())
    _check_attention(b, o, lse, seen)
    # wider masks than the sequences need
    wide = torch.cat([masks, torch.full((2 * n, 4), -1, dtype=torch.int32)], 1)
    o2, lse2 = _attend(tpa, b, None, wide.cuda())
    assert torch.equal(o[:2 * n], o2[:2 * n])


@pytest.mark.parametrize("n", [8, 60])
def test_positions_out_of_place_are_held(tpa, n):
    b = Batch([n], [400], 4, 1, 64, 32, seed=37)
    trees = _trees([n], 9)
    positions, masks = tpa.draft_masks(_flat(trees).cuda(), b.offsets, b.kv_lens, n, 50)
    chain = torch.arange(400 - n, 400, dtype=torch.int32).cuda()
    for wrong, right in ((torch.full_like(positions, -5), torch.full_like(positions, 400 - n)),
                         (torch.full_like(positions, 2 ** 31 - 1), chain)):
        a = _attend(tpa, b, wrong, masks, 50)
        c = _attend(tpa, b, right, masks, 50)
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


@pytest.mark.parametrize("n", [8, 50])
def test_slots_behind_the_sequence_may_hold_anything(tpa, n):
    b = Batch([n, n], [n + 37, 500], 8, 2, 128, 16, seed=38)
    trees = _trees([n, n], 9)
    positions, masks = tpa.draft_masks(_flat(trees).cuda(), b.offsets, b.kv_lens, n)
    want = _attend(tpa, b, positions, masks)
    used = torch.zeros(b.k_cache.shape[0], b.page, dtype=torch.bool)
    for s, kv in enumerate(b.kv_lens_list):
        j = torch.arange(kv)
        used[torch.tensor(b.rows[s])[j // b.page], j % b.page] = True
    for c in (b.k_cache, b.v_cache):
        c.transpose(1, 2)[~used.cuda()] = float("nan")
    got = _attend(tpa, b, positions, masks)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_a_sequence_with_too_many_tokens_is_reported(tpa):
    b = Batch([3, 40, 2], [30, 80, 200], 4, 1, 64, 16, seed=39)
    trees = _trees(b.q_lens, 2)
    _, masks = tpa.draft_masks(_flat(trees).cuda(), b.offsets, b.kv_lens, 64)
    o = torch.full_like(b.q, 7.0)
    lse = torch.full(b.q.shape[:2], 7.0, device="cuda")
    tpa.paged_attn_tree_fwd(*b.cache, b.q, masks[:, :1].contiguous(), max_q_len=40, out=o, lse=lse)
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()
    assert (o[3:43] == 7.0).all() and (lse[3:43] == 7.0).all()
    seen = _seen(trees, b.kv_lens_list)
    for s, rows in ((0, slice(0, 3)), (2, slice(43, 45))):
        ref, _, size = attend_tree(b.q[rows].cpu(), b.sequence(s, b.k_cache), b.sequence(s, b.v_cache), seen[s])
        assert ((o[rows].double().cpu() - ref).abs() <= (2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * ref.abs()).all()


# ------------------------------------------------------------------ accepted paths

@pytest.mark.parametrize("form", ["wide", "chain", "loose", "star"])
@pytest.mark.parametrize("q_lens", [[1], [0, 5, 1], [16, 64, 33, 0, 7], [1024, 300]])
@pytest.mark.parametrize("most", [1, 3, 40, 1024])
def test_accept(tpa, q_lens, form, most):
    trees = _trees(q_lens, 11, form)
    r = np.random.default_rng(4)
    n = sum(q_lens)
    drafted, sampled = r.integers(0, 3, n), r.integers(0, 3, n)  # few tokens: equal children, long paths
    if form == "chain":
        sampled = np.where(r.random(n) < 0.97, np.roll(drafted, -1), 5)
    S = len(q_lens)
    outs = [guarded(s, torch.int32) for s in ((S, most), (S, most), (S,))]
    tpa.accept_drafts(_flat(trees).cuda(), _i32([0] + list(np.cumsum(q_lens))).cuda(), _i32(drafted).cuda(),
                      _i32(sampled).cuda(), most, out=tuple(o for _, o in outs))
    for buf, _ in outs:
        check_guards(buf, "out")
    tokens, path, count = (o.cpu() for _, o in outs)
    at = 0
    for s, t in enumerate(trees):
        rows, emitted = accept(t, drafted[at:at + len(t)].tolist(), sampled[at:at + len(t)].tolist(), most)
        assert count[s] == len(rows)
        assert path[s].tolist() == rows + [-1] * (most - len(rows))
        assert tokens[s].tolist() == emitted + [-1] * (most - len(rows))
        at += len(t)
    tpa.sync_status()


def _compacted(b, cache, paths):
    """The cache after the paths' tokens have moved, read before any is written."""
    out = cache.clone()
    for s, path in enumerate(paths):
        base = b.kv_lens_list[s] - b.q_lens[s]
        at = lambda slot: (b.rows[s][slot // b.page], slot % b.page)  # noqa: E731
        for i, p in enumerate(path):
            (fp, fs), (tp, ts) = at(base + p), at(base + i)
            out[..., tp, :, ts, :] = cache[..., fp, :, fs, :]
    return out


@pytest.mark.parametrize("layers", [None, 1, 3])
@pytest.mark.parametrize("q_lens,kv_lens,hkv,d,page", [([1], [1], 1, 64, 16), ([20, 0, 7, 33], [20, 5, 300, 64], 8, 128, 16),
                                                       ([64, 12], [130, 1000], 2, 64, 128), ([300], [400], 3, 128, 32),
                                                       ([9], [777], 40, 128, 64)])
def test_compact(tpa, q_lens, kv_lens, hkv, d, page, layers):
    b = Batch(q_lens, kv_lens, hkv, hkv, d, page, seed=41)
    r = np.random.default_rng(6)
    paths = []
    for n in q_lens:
        keep = np.nonzero(r.random(n) < 0.4)[0].tolist()
        paths.append(([0] if n else []) + [k for k in keep if k > 0])
    most = max(1, max(len(p) for p in paths))
    path = _i32([p + [-1] * (most - len(p)) for p in paths]).cuda()
    count = _i32([len(p) for p in paths]).cuda()
    kc, vc = b.k_cache, b.v_cache
    if layers:
        g = torch.Generator().manual_seed(1)
        kc, vc = (torch.randn((layers, *b.k_cache.shape), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    want = _compacted(b, kc.cpu(), paths), _compacted(b, vc.cpu(), paths)
    lens = tpa.paged_compact(kc, vc, b.pages, b.offsets, b.kv_lens, path, count)
    tpa.sync_status()
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])
    assert lens.tolist() == [k - q + len(p) for k, q, p in zip(kv_lens, q_lens, paths)]


def test_compact_leaves_what_is_no_path(tpa):
    b = Batch([10, 10], [100, 200], 2, 2, 64, 16, seed=43)
    before = b.k_cache.clone(), b.v_cache.clone()
    for path, n in (([0, 2, 2], 3), ([0, 10, -1], 2), ([1, 0, -1], 2), ([0, 3, 5], 4), ([0, 3, 5], -1), ([-1, 3, 5], 2)):
        lens = tpa.paged_compact(b.k_cache, b.v_cache, b.pages, b.offsets, b.kv_lens, _i32([path, [0, 1, 2]]).cuda(),
                                 _i32([n, 3]).cuda())
        with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
            tpa.sync_status()
        assert lens.tolist() == [100, 193]
        assert torch.equal(b.k_cache, before[0]) and torch.equal(b.v_cache, before[1])
    # a page out of range where a token moves from: only that token stays
    b.pages[0, 93 // 16] = 10 ** 6
    tpa.paged_compact(b.k_cache, b.v_cache, b.pages, b.offsets, b.kv_lens, _i32([[0, 3], [0, 1]]).cuda(), _i32([2, 2]).cuda())
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()
    assert torch.equal(b.k_cache, before[0])


def test_compact_past_32_bits(tpa):
    """Layers whose bytes pass 2^32."""
    b = Batch([5], [40], 8, 8, 128, 16, seed=44)
    n_pages = 70000
    kc = torch.zeros((3, n_pages, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    b.pages[0, 2] = n_pages - 1
    for layer in range(3):
        kc[layer, n_pages - 1, :, 3:8] = torch.arange(5, device="cuda").view(1, 5, 1).to(torch.bfloat16) + 10 * layer
        vc[layer, n_pages - 1, :, 3:8] = -1 - torch.arange(5, device="cuda").view(1, 5, 1).to(torch.bfloat16)
    tpa.paged_compact(kc, vc, b.pages, b.offsets, b.kv_lens, _i32([[0, 2, 4]]).cuda(), _i32([3]).cuda())
    tpa.sync_status()
    for layer in range(3):
        assert kc[layer, n_pages - 1, 5, 3:8, 7].tolist() == [10 * layer + x for x in (0, 2, 4, 3, 4)]
        assert vc[layer, n_pages - 1, 0, 3:8, 100].tolist() == [-1 - x for x in (0, 2, 4, 3, 4)]


def test_a_round_together_captured(tpa):
    """Masks, rotation at the tree's positions, append, attention, sampling, the accepted path and the compacted cache, once
    captured and replayed while the sequences grow; each round's tokens are those of attention over the
    accepted tokens alone, one sequence at a time."""
    S, n, hq, hkv, d, page, vocab = 3, 12, 8, 2, 64, 16, 50
    g = torch.Generator().manual_seed(50)
    rand = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    table = tpa.rope_table(400, d)
    embed, wq, wk, wv, head = rand(vocab, 64), 0.3 * rand(64, hq * d), 0.3 * rand(64, hkv * d), rand(64, hkv * d), rand(hq * d, vocab)
    kc, vc = rand(60, hkv, page, d), rand(60, hkv, page, d)
    pages = torch.randperm(60, generator=g).to(torch.int32)[:S * 20].view(S, 20).contiguous().cuda()
    lens = _i32([40, 1 + 0, 17]).cuda()                    # committed tokens
    offsets = _i32([n * s for s in range(S + 1)]).cuda()
    trees = _trees([n] * S, 8)
    parents = _flat(trees).cuda()
    drafted = torch.zeros(S * n, dtype=torch.int32, device="cuda")
    u = torch.zeros(S * n, device="cuda")

    barred = torch.arange(vocab, device="cuda") >= 4   # few tokens may be drawn, so that drafts among them fit

    def step():
        kv = lens + n
        positions, masks = tpa.draft_masks(parents, offsets, kv, n)
        x = embed[drafted.long()]
        q, k, v = (x @ wq).view(-1, hq, d), (x @ wk).view(-1, hkv, d), (x @ wv).view(-1, hkv, d)
        q, k = tpa.qk_norm_rope_fwd(positions, q, k, table)
        tpa.paged_append(kc, vc, pages, offsets, kv, k, v)
        o, _ = tpa.paged_attn_tree_fwd(kc, vc, pages, offsets, kv, q, masks, max_q_len=n)
        logits = (o.view(-1, hq * d) @ head).masked_fill(barred, float("-inf"))
        sampled, logp = tpa.sample_tokens(logits, u, 0.9, 20, 0.95)
        tokens, path, count = tpa.accept_drafts(parents, offsets, drafted, sampled, n)
        lens.copy_(tpa.paged_compact(kc, vc, pages, offsets, kv, path, count))
        return sampled, tokens, path, count, logits

    def inputs():
        drafted.copy_(torch.randint(0, 3, (S * n,), generator=g))   # few tokens: some fit
        u.copy_(torch.rand(S * n, generator=g))

    history = [(c[pages[s].long()][:, :, :].transpose(1, 2).reshape(-1, hkv, d)[:int(lens[s])].clone()) for s in range(S) for c in (kc, vc)]
    inputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved = lens.clone(), kc.clone(), vc.clone()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for a, z in zip((lens, kc, vc), saved):
        a.copy_(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sampled, tokens, path, count, logits = step()
    accepted = 0
    for _ in range(6):
        inputs()
        before = lens.clone()
        graph.replay()
        torch.cuda.synchronize()
        tpa.sync_status()
        assert torch.equal(lens, before + count)
        for s in range(S):
            rows = path[s, :int(count[s])].long()
            want, emitted = accept(trees[s], drafted[s * n:(s + 1) * n].tolist(), sampled[s * n:(s + 1) * n].tolist(), n)
            assert rows.tolist() == want and tokens[s, :len(want)].tolist() == emitted
            accepted += len(want) - 1
            # the accepted tokens as a chain behind the sequence's history
            x = embed[drafted[s * n + rows].long()]
            pos = torch.arange(int(before[s]), int(before[s]) + len(want), dtype=torch.int32, device="cuda")
            q, k = tpa.qk_norm_rope_fwd(pos, (x @ wq).view(-1, hq, d), (x @ wk).view(-1, hkv, d), table)
            v = (x @ wv).view(-1, hkv, d)
            history[2 * s], history[2 * s + 1] = torch.cat([history[2 * s], k]), torch.cat([history[2 * s + 1], v])
            cached = [c[pages[s].long()].transpose(1, 2).reshape(-1, hkv, d)[:int(lens[s])] for c in (kc, vc)]
            assert torch.equal(cached[1], history[2 * s + 1])
            assert (cached[0].float() - history[2 * s].float()).abs().max() <= 2.0 ** -6 * history[2 * s].float().abs().max()
            kv = cached[0].shape[0]
            seen = torch.arange(kv)[None] <= torch.arange(kv - len(want), kv)[:, None]
            ref, _, size = attend_tree(q.cpu(), cached[0].cpu(), cached[1].cpu(), seen)
            o = ref.reshape(len(want), -1).to(torch.bfloat16).float() @ head.cpu().float()
            got = logits[s * n + rows].float().cpu()
            # O off by 2^-7 of its size, the head's products and its logits' rounding: a small share of their size
            bound = 2.0 ** -6 * (size.reshape(len(want), -1).float() @ head.cpu().float().abs()) + 2.0 ** -6 * o.abs()
            assert ((got - o).abs() <= bound)[:, :4].all() and torch.isinf(got[:, 4:]).all()
    assert accepted > 0
