"""Calls of the sampling step's operators that have to be refused, or taken as
no work, before anything is launched (CPU)."""
import ctypes as C
import math

import pytest
import torch

P = 4096  # an aligned address that no such call follows
INVALID = -1


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    return tpa


def _i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def _sample(L, logits=P, kind=0, stride=100, rows=2, vocab=100, u=P, tokens=P, logp=P, none=False, **kw):
    from prefix_shared_tree_attention_gb300._abi import SampleParams
    p = SampleParams(None, None, None, None, 1.0, 1.0, 0.0, 0)
    for k, v in kw.items():
        setattr(p, k, v)
    return L.tpa_sample_tokens(logits, kind, stride, rows, vocab, None if none else C.byref(p), u, tokens, logp, None)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(vocab=0), dict(vocab=2 ** 30 + 1), dict(kind=2), dict(kind=-1), dict(none=True),
                                dict(temperature_all=-1.0), dict(temperature_all=1e-7), dict(temperature_all=1e7),
                                dict(temperature_all=math.nan), dict(temperature_all=math.inf), dict(top_p_all=-0.1),
                                dict(top_p_all=1.1), dict(top_p_all=math.nan), dict(min_p_all=-0.1), dict(min_p_all=2.0),
                                dict(min_p_all=math.nan), dict(logits=None), dict(u=None), dict(tokens=None), dict(logp=None),
                                dict(stride=99), dict(stride=2 ** 41), dict(logits=P + 2), dict(kind=1, logits=P + 1), dict(u=P + 2),
                                dict(tokens=P + 1), dict(logp=P + 2), dict(temperature=P + 2), dict(top_k=P + 1)])
def test_sample_refusals(tpa, kw):
    assert _sample(tpa.lib(), **kw) == INVALID


def test_no_rows_are_no_work(tpa):
    assert _sample(tpa.lib(), rows=0, logits=None, u=None, tokens=None, logp=None) == 0


def test_sample_arguments(tpa):
    x, u = torch.zeros((3, 8)), torch.zeros(3)
    for bad in (dict(logits=x.double()), dict(logits=x.half()), dict(logits=x[0]), dict(logits=torch.zeros((8, 3)).t()),
                dict(u=u[:2]), dict(u=u.double()), dict(temperature=torch.ones(2)), dict(temperature=torch.ones(3).double()),
                dict(top_k=torch.ones(3)), dict(top_p=torch.ones(6)[::2]), dict(top_k=2 ** 31), dict(top_k=-2 ** 40)):
        with pytest.raises(ValueError):
            tpa.sample_tokens(**{**dict(logits=x, u=u), **bad})
    with pytest.raises(ValueError, match="CUDA"):
        tpa.sample_tokens(x, u)


def _view(**kw):
    from prefix_shared_tree_attention_gb300._abi import PagedView
    v = PagedView()
    v.k_cache = v.v_cache = v.pages = v.offsets = v.kv_lens = P
    v.n_pages, v.page_size, v.n_seqs, v.max_pages, v.page_stride = 10, 16, 2, 4, 4
    v.n_heads_kv, v.head_dim, v.n_rows = 2, 64, 3
    for k, x in kw.items():
        setattr(v, k, x)
    return v


def _tree(L, masks=P, words=1, positions=P, window=0, view=None):
    return L.tpa_paged_attn_tree_fwd(C.byref(view or _view()), P, 256, masks, words, positions, P, P, 4, 3, 0.0, window, None, 0, None)


@pytest.mark.parametrize("kw", [dict(masks=None), dict(words=0), dict(words=33), dict(words=-1), dict(masks=P + 2), dict(positions=P + 1),
                                dict(positions=None, window=5), dict(window=-1), dict(view=dict(head_dim=96)),
                                dict(view=dict(page_size=8)), dict()])  # the last: no workspace
def test_tree_attention_refusals(tpa, kw):
    kw = dict(kw)
    if "view" in kw:
        kw["view"] = _view(**kw["view"])
    assert _tree(tpa.lib(), **kw) == INVALID


def test_tree_attention_without_rows(tpa):
    assert _tree(tpa.lib(), masks=None, positions=None, view=_view(n_rows=0)) == 0


def test_tree_attention_arguments(tpa):
    bf = torch.bfloat16
    cache = torch.zeros((3, 2, 16, 64), dtype=bf)
    call = dict(k_cache=cache, v_cache=cache.clone(), pages=_i32(2, 3), offsets=_i32(3), kv_lens=_i32(2),
                q=torch.zeros((4, 4, 64), dtype=bf), max_q_len=2, masks=_i32(4, 1))
    for bad in (dict(masks=_i32(3, 1)), dict(masks=_i32(4)), dict(masks=torch.zeros((4, 1))), dict(masks=_i32(4, 33)), dict(masks=_i32(4, 0)),
                dict(masks=_i32(4, 2)[:, :1]), dict(positions=_i32(3)), dict(positions=torch.zeros(4)), dict(window=3),
                dict(window=-1), dict(max_q_len=2 ** 31), dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 26))):
        with pytest.raises(ValueError):
            tpa.paged_attn_tree_fwd(**{**call, **bad})
    with pytest.raises(ValueError, match="CUDA"):
        tpa.paged_attn_tree_fwd(**call)


def _masks(L, parents=P, offsets=P, lens=P, seqs=2, rows=4, window=0, positions=P, masks=P, words=1):
    return L.tpa_draft_masks(parents, offsets, lens, seqs, rows, window, positions, masks, words, None)


@pytest.mark.parametrize("kw", [dict(parents=None), dict(offsets=None), dict(lens=None), dict(seqs=-1), dict(rows=-1), dict(rows=2 ** 30),
                                dict(window=-1), dict(positions=None), dict(masks=None), dict(words=0), dict(words=33), dict(seqs=0),
                                dict(parents=P + 2), dict(masks=P + 1)])
def test_masks_refusals(tpa, kw):
    assert _masks(tpa.lib(), **kw) == INVALID


def _accept(L, parents=P, offsets=P, drafted=P, sampled=P, seqs=2, rows=4, tokens=P, path=P, count=P, most=3):
    return L.tpa_accept_drafts(parents, offsets, drafted, sampled, seqs, rows, tokens, path, count, most, None)


@pytest.mark.parametrize("kw", [dict(parents=None), dict(offsets=None), dict(drafted=None), dict(sampled=None), dict(seqs=-1), dict(rows=-1),
                                dict(rows=2 ** 30), dict(tokens=None), dict(path=None), dict(count=None), dict(most=0), dict(most=1025),
                                dict(seqs=0), dict(path=P + 2)])
def test_accept_refusals(tpa, kw):
    assert _accept(tpa.lib(), **kw) == INVALID


def test_empty_batches_are_no_work(tpa):
    L = tpa.lib()
    assert _masks(L, None, None, None, 0, 0, 0, None, None) == 0
    assert _accept(L, None, None, None, None, 0, 0, None, None, None) == 0
    assert L.tpa_paged_compact(C.byref(_view(n_seqs=0, n_rows=0)), 1, None, None, 1, None, None) == 0


@pytest.mark.parametrize("kw", [dict(layers=0), dict(layers=32768), dict(path=None), dict(count=None), dict(lens=None), dict(lens=P),
                                dict(most=0), dict(path=3 * P + 2), dict(view=dict(pages=None)), dict(view=dict(n_pages=0)),
                                dict(view=dict(k_cache=P + 8))])
def test_compact_refusals(tpa, kw):
    a = {**dict(layers=1, path=3 * P, count=3 * P, lens=2 * P, most=3), **kw}
    assert tpa.lib().tpa_paged_compact(C.byref(_view(**a.get("view", {}))), a["layers"], a["path"], a["count"], a["most"], a["lens"],
                                       None) == INVALID


def test_draft_arguments(tpa):
    par, off, lens = _i32(4), _i32(3), _i32(2)
    for bad in (dict(max_q_len=0), dict(max_q_len=1025), dict(max_q_len=2 ** 33), dict(window=-1), dict(parents=torch.zeros(4)),
                dict(offsets=_i32(4)), dict(kv_lens=_i32(4)[::2])):
        with pytest.raises(ValueError):
            tpa.draft_masks(**{**dict(parents=par, offsets=off, kv_lens=lens, max_q_len=4), **bad})
    for bad in (dict(max_path=0), dict(max_path=1025), dict(draft_tokens=_i32(3)), dict(sampled=_i32(4).long()),
                dict(out=(_i32(2, 3), _i32(2, 3), _i32(3)))):
        with pytest.raises(ValueError):
            tpa.accept_drafts(**{**dict(parents=par, offsets=off, draft_tokens=_i32(4), sampled=_i32(4), max_path=3), **bad})
    cache = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    call = dict(k_cache=cache, v_cache=cache.clone(), pages=_i32(2, 3), offsets=off, kv_lens=lens, path=_i32(2, 3), n_accepted=_i32(2))
    for bad in (dict(k_cache=cache.float()), dict(k_cache=cache[0]), dict(v_cache=cache[:2]), dict(path=_i32(3, 3)), dict(n_accepted=_i32(3)),
                dict(path=_i32(6)), dict(out=_i32(3)), dict(k_cache=cache[None, None], v_cache=cache[None, None]),
                dict(k_cache=torch.zeros((0, 3, 2, 16, 64), dtype=torch.bfloat16), v_cache=torch.zeros((0, 3, 2, 16, 64), dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            tpa.paged_compact(**{**call, **bad})
    with pytest.raises(ValueError, match="CUDA"):
        tpa.paged_compact(**call)


def _pool(**kw):
    from prefix_shared_tree_attention_gb300._abi import PagedPool
    v = PagedPool()
    v.k_cache = v.v_cache = v.pages = v.kv_lens = v.refs = P
    v.n_layers, v.n_pages, v.page_size, v.n_heads_kv, v.head_dim, v.n_seqs, v.max_pages, v.page_stride = 1, 10, 16, 2, 64, 2, 4, 4
    for k, x in kw.items():
        setattr(v, k, x)
    return v


BAD_POOLS = [dict(refs=None), dict(pages=None), dict(kv_lens=None), dict(n_pages=0), dict(page_size=8), dict(n_seqs=-1), dict(max_pages=-1),
             dict(page_stride=3), dict(max_pages=2 ** 26, page_stride=2 ** 26), dict(refs=P + 2), dict(pages=P + 1)]


@pytest.mark.parametrize("kw", BAD_POOLS + [dict(n_seqs=8193)])
def test_resize_refusals(tpa, kw):
    assert tpa.lib().tpa_paged_resize(C.byref(_pool(**kw)), P, None) == INVALID
    assert tpa.lib().tpa_paged_resize(None, P, None) == INVALID and tpa.lib().tpa_paged_resize(C.byref(_pool()), None, None) == INVALID


@pytest.mark.parametrize("kw", BAD_POOLS + [dict(k_cache=None), dict(v_cache=None), dict(k_cache=P + 8), dict(n_layers=0),
                                            dict(n_layers=32768), dict(head_dim=96), dict(n_heads_kv=0), dict(n_heads_kv=65536),
                                            dict(n_pages=2 ** 27), dict(n_seqs=2 ** 18 + 1)])
def test_fork_refusals(tpa, kw):
    assert tpa.lib().tpa_paged_fork(C.byref(_pool(**kw)), P, P, 1, P, None) == INVALID


@pytest.mark.parametrize("args", [(None, P, 1, P), (P, None, 1, P), (P, P, -1, P), (P, P, 8193, P), (P, P, 1, None), (P + 1, P, 1, P)])
def test_fork_list_refusals(tpa, args):
    assert tpa.lib().tpa_paged_fork(C.byref(_pool()), *args, None) == INVALID


def test_pool_arguments(tpa):
    pages, lens, refs = _i32(2, 3), _i32(2), _i32(5)
    cache = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    for bad in (dict(pages=pages.long()), dict(pages=_i32(3, 2).t()), dict(kv_lens=_i32(3)), dict(refs=_i32(5, 1)), dict(refs=torch.zeros(5)),
                dict(page_size=2 ** 32 + 16), dict(out=_i32(2))):
        with pytest.raises(ValueError):
            tpa.paged_resize(**{**dict(pages=pages, kv_lens=lens, refs=refs, page_size=16), **bad})
    for bad in (dict(src=_i32(2)), dict(src=_i32(1, 1)), dict(dst=torch.zeros(1)), dict(refs=_i32(4)), dict(k_cache=cache.float()),
                dict(v_cache=cache[:4])):
        with pytest.raises(ValueError):
            tpa.paged_fork(**{**dict(k_cache=cache, v_cache=cache.clone(), pages=pages, kv_lens=lens, refs=refs, src=_i32(1),
                                     dst=_i32(1)), **bad})
    with pytest.raises(ValueError, match="CUDA"):
        tpa.paged_resize(pages, lens, refs, 16)


def test_compact_lengths_are_not_the_accepted_numbers(tpa):
    assert tpa.lib().tpa_paged_compact(C.byref(_view()), 1, 3 * P, 4 * P, 3, 4 * P, None) == INVALID


def test_vocabularies_have_a_limit(tpa):
    assert _sample(tpa.lib(), vocab=2 ** 24 + 1, stride=2 ** 25) == INVALID
    assert _sample(tpa.lib(), vocab=2 ** 24, stride=2 ** 25, rows=0) == 0
