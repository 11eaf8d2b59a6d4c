"""GPU parity of the paged append (tpa_paged_append): the rows written against
fp64 (tolerances as in test_gpu_rope.py), every other byte of the cache and of
q_out as it was."""
import pytest
import torch

from oracle.rope import norm_rope
from _paged import Batch
from _pipeline import check_guards, guarded

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _check(tpa, b, table, wq, wk, inter=False, with_q=True):
    bk, kc = guarded(b.k_cache.shape, torch.bfloat16)
    bv, vc = guarded(b.v_cache.shape, torch.bfloat16)
    kc.copy_(b.k_cache)
    vc.copy_(b.v_cache)
    bq, qo = guarded(b.q.shape, torch.bfloat16)
    qo.fill_(7.0)
    got = tpa.paged_append(kc, vc, b.pages, b.offsets, b.kv_lens, b.k, b.v, q=b.q if with_q else None, table=table,
                           q_weight=wq, k_weight=wk, eps=EPS, interleaved=inter, q_out=qo if with_q else None)
    for buf, what in ((bk, "k_cache"), (bv, "v_cache"), (bq, "q_out")):
        check_guards(buf, what)
    n = b.total
    _, pos = b.places()
    row = None if table is None else table.cpu()[pos]
    page, slot = b.slots()
    kc_, vc_ = kc.cpu(), vc.cpu()
    for x, w, y in ((b.k, wk, kc_[page, :, slot]), (b.q, wq, qo.cpu()[:n])):
        if x is b.q and not with_q:
            assert got is None and (qo == 7.0).all()
            continue
        ref, size = norm_rope(x.cpu()[:n], None if w is None else w.cpu(), row, EPS, inter)
        off = (y.double() - ref).abs() - (2.0 ** -19 * size * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs())
        assert n == 0 or off.max() <= 0
    assert torch.equal(vc_[page, :, slot], b.v.cpu()[:n])
    if with_q:
        assert (qo[n:] == 7.0).all()
    written = torch.zeros(kc.shape[0], kc.shape[2], dtype=torch.bool)
    written[page, slot] = True
    keep = ~written[:, None, :, None].expand(kc.shape)
    assert torch.equal(kc_[keep], b.k_cache.cpu()[keep]) and torch.equal(vc_[keep], b.v_cache.cpu()[keep])


CASES = [  # q_lens, kv_lens, hq, hkv, d, page, extra rows
    ([1], [1], 1, 1, 64, 16, 0), ([1] * 9, [1, 16, 17, 33, 5, 100, 64, 65, 2], 32, 8, 128, 16, 3),
    ([5, 0, 1, 300, 0], [5, 40, 129, 300, 0], 8, 2, 128, 64, 10), ([70, 33], [170, 33], 10, 5, 64, 32, 0),
    ([1] * 100, list(range(1, 101)), 3, 1, 128, 128, 28), ([0, 0, 3], [0, 9, 3], 4, 4, 64, 16, 1),
    ([257], [1000], 33, 11, 64, 128, 0), ([500, 1, 90], [500, 700, 130], 16, 4, 128, 64, 5),
    ([900], [900], 20, 20, 128, 16, 3), ([999, 1, 1], [999, 1, 30], 1, 1, 128, 32, 40)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("rot,inter,norm,with_q", [(1, False, True, True), (2, True, False, True), (0, False, True, False),
                                                   (0, False, False, True)])
def test_append(tpa, case, rot, inter, norm, with_q):
    b = Batch(*case[:6], seed=17, extra=case[6])
    g = torch.Generator().manual_seed(1)
    wq, wk = ((1 + 0.3 * torch.randn(b.d, generator=g)).cuda() for _ in range(2)) if norm else (None, None)
    table = tpa.rope_table(1000, b.d // rot) if rot else None
    _check(tpa, b, table, wq, wk, inter, with_q)
    tpa.sync_status()


def test_slices_of_a_fused_projection(tpa):
    b = Batch([3, 4], [10, 4], 4, 2, 128, 16, seed=2)
    qkv = torch.randn((7, 8 * 128), device="cuda").to(torch.bfloat16)
    b.q, b.k, b.v = qkv[:, :512].view(7, 4, 128), qkv[:, 512:768].view(7, 2, 128), qkv[:, 768:].view(7, 2, 128)
    _check(tpa, b, tpa.rope_table(10, 128), None, None)


@pytest.mark.parametrize("hq,hkv,extra", [(4, 2, 0), (8, 4, 1100)])  # few bytes and many: other kernels
def test_bad_batches_are_reported_and_skipped(tpa, hq, hkv, extra):
    table = tpa.rope_table(64, 64)

    def run(change, skipped, moved=()):
        b = Batch([2, 3, 1], [20, 3, 33], hq, hkv, 64, 16, seed=5, extra=extra)
        good = b.k_cache.clone(), b.v_cache.clone()
        want = tpa.paged_append(*good, b.pages, b.offsets, b.kv_lens, b.k, b.v, q=b.q, table=table)
        page, slot = b.slots()
        change(b)
        got = torch.full_like(b.q, 7.0)
        tpa.paged_append(*b.cache, b.k, b.v, q=b.q, table=table, q_out=got)
        with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
            tpa.sync_status()
        tpa.sync_status()
        keep = [i for i in range(6) if i not in skipped and i not in moved]
        assert torch.equal(got[keep], want[keep]) and (got[sorted(skipped)] == 7.0).all() and (got[6:] == 7.0).all()
        for c, w in zip((b.k_cache, b.v_cache), good):
            assert torch.equal(c[page, :, slot][keep], w[page, :, slot][keep])

    def page_of(s, i, value):
        def f(b):
            b.pages[s, i] = value
        return f

    def length(s, value):
        def f(b):
            b.kv_lens[s] = value
        return f

    run(page_of(0, 1, -1), {0, 1})
    run(page_of(0, 1, 2 ** 31 - 1), {0, 1})
    run(page_of(1, 0, 1000), {2, 3, 4})
    run(length(1, 2), {2}, {3, 4})               # its first token would be at position -1, the others are at 0 and 1
    run(length(1, -2 ** 31), {2, 3, 4})
    run(length(2, 2 ** 31 - 1), {5})
    run(length(2, 49), {5})                      # more tokens than the pages hold


def test_positions_past_the_table(tpa):
    b = Batch([2], [20], 4, 2, 64, 16, seed=5)
    before = b.k_cache.clone()
    tpa.paged_append(*b.cache, b.k, b.v, table=tpa.rope_table(18, 64))
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()
    assert torch.equal(before, b.k_cache)


@pytest.mark.parametrize("hq,hkv,extra", [(4, 2, 0), (8, 4, 1100)])
def test_unordered_offsets_end_and_stay_inside(tpa, hq, hkv, extra):
    # no promise but that nothing outside the tensors is touched and the call is reported or skipped
    for off in ([0, 5, 2, 6], [3, 3, 3, 3], [0, 2, 5, 1000], [-7, 2, 5, 6], [6, 5, 2, 0], [0, 2 ** 31 - 1, -2 ** 31, 6]):
        b = Batch([2, 3, 1], [20, 3, 33], hq, hkv, 64, 16, seed=5, extra=extra)
        b.offsets.copy_(torch.tensor(off, dtype=torch.int32))
        bk, kc = guarded(b.k_cache.shape, torch.bfloat16)
        bv, vc = guarded(b.v_cache.shape, torch.bfloat16)
        kc.copy_(b.k_cache)
        vc.copy_(b.v_cache)
        bq, qo = guarded(b.q.shape, torch.bfloat16)
        tpa.paged_append(kc, vc, b.pages, b.offsets, b.kv_lens, b.k, b.v, q=b.q, q_out=qo)
        try:
            tpa.sync_status()
        except tpa.TpaError as e:
            assert e.name == "TPA_ERR_INVALID_ARG"
        for buf, what in ((bk, "k_cache"), (bv, "v_cache"), (bq, "q_out")):
            check_guards(buf, what)


def test_a_cache_past_32_bits(tpa):
    # 5.4 GB for the keys: the last page's rows are past 2^32 bytes
    n_pages, hkv, page, d = 20480, 8, 128, 128
    kc = torch.zeros((n_pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros((n_pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    b = Batch([2, 2], [130, 2], 8, hkv, d, page, seed=3)
    pages = torch.tensor([[5, n_pages - 1], [n_pages // 2 + 1, 0]], dtype=torch.int32, device="cuda")
    tpa.paged_append(kc, vc, pages, b.offsets, b.kv_lens, b.k, b.v)
    tpa.sync_status()
    for c, x in ((kc, b.k), (vc, b.v)):
        assert torch.equal(c[n_pages - 1, :, 0:2].transpose(0, 1), x[:2])
        assert torch.equal(c[n_pages // 2 + 1, :, 0:2].transpose(0, 1), x[2:])
        assert int((c != 0).sum()) == int((x != 0).sum())


def test_graph_replayed_over_a_growing_sequence(tpa):
    b = Batch([1, 1], [40, 7], 4, 2, 64, 16, seed=4, spare=0)
    b.kv_lens.copy_(torch.tensor([37, 4], dtype=torch.int32))
    table = tpa.rope_table(64, 64)
    eager = b.k_cache.clone(), b.v_cache.clone()
    q_out = torch.empty_like(b.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tpa.paged_append(*b.cache, b.k, b.v, q=b.q, table=table, q_out=q_out)
    lens = b.kv_lens.clone()
    for step in range(3):
        b.k.normal_()
        b.v.normal_()
        b.q.normal_()
        b.kv_lens.copy_(lens + step)
        want = tpa.paged_append(*eager, b.pages, b.offsets, b.kv_lens, b.k, b.v, q=b.q, table=table)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, want) and torch.equal(eager[0], b.k_cache) and torch.equal(eager[1], b.v_cache)
    tpa.sync_status()
