"""Calls of the policy's operators that have to be refused, or taken as no
work, before anything is launched (CPU)."""
import ctypes as C

import pytest
import torch

P = 4096  # an aligned address that no such call follows


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    return tpa


def _view(**kw):
    from prefix_shared_tree_attention_gb300._abi import PagedView
    v = PagedView()
    v.k_cache = v.v_cache = v.pages = v.offsets = v.kv_lens = P
    v.n_pages, v.page_size, v.n_seqs, v.max_pages, v.page_stride = 10, 16, 2, 4, 4
    v.n_heads_kv, v.head_dim, v.n_rows = 2, 64, 0
    for k, x in kw.items():
        setattr(v, k, x)
    return v


NONE = [dict(n_seqs=0), dict(n_seqs=0, pages=None, kv_lens=None), dict(n_seqs=0, pages=None, kv_lens=None, max_pages=0, page_stride=0)]


def _append(L, view):
    from prefix_shared_tree_attention_gb300._abi import RopeParams
    return L.tpa_paged_append(C.byref(view), None, 128, None, 128, None, 0, None, 0, 0, C.byref(RopeParams()), None)


def _attend(L, view, max_q=1):
    return L.tpa_paged_attn_fwd(C.byref(view), None, 256, None, None, 4, max_q, 0.0, 0, None, 0, None)


@pytest.mark.parametrize("kw", NONE)
def test_no_sequences_are_no_work(tpa, kw):
    assert _append(tpa.lib(), _view(**kw)) == 0
    assert _attend(tpa.lib(), _view(**kw)) == 0 and _attend(tpa.lib(), _view(**kw), max_q=0) == 0


@pytest.mark.parametrize("kw", [dict(n_seqs=0, n_rows=1), dict(n_seqs=-1), dict(n_seqs=0, k_cache=None), dict(n_seqs=0, page_size=8),
                                dict(n_seqs=0, offsets=None), dict(n_seqs=0, max_pages=-1), dict(max_pages=0), dict(pages=None)])
def test_other_views_stay_refused(tpa, kw):
    assert _append(tpa.lib(), _view(**kw)) == -1 and _attend(tpa.lib(), _view(**kw)) == -1


def test_most_new_tokens_below_zero(tpa):
    assert _attend(tpa.lib(), _view(), max_q=-1) == -1 and _attend(tpa.lib(), _view(n_rows=1), max_q=0) == -1


@pytest.fixture
def call():
    bf = torch.bfloat16
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    cache = torch.zeros((3, 2, 16, 64), dtype=bf)
    return dict(k_cache=cache, v_cache=cache.clone(), pages=i32(2, 3), offsets=i32(3), kv_lens=i32(2),
                q=torch.zeros((4, 4, 64), dtype=bf), max_q_len=2)


def test_a_workspace_has_all_its_bytes(tpa, call):
    # a broadcast byte has as many elements as are asked for, and memory for one
    ws = torch.zeros(1, dtype=torch.uint8).expand(1 << 26)
    with pytest.raises(ValueError, match="workspace"):
        tpa.paged_attn_fwd(**call, workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        tpa.paged_attn_fwd(**call, workspace=torch.zeros(1 << 20, dtype=torch.uint8)[::2])
    q, k = torch.zeros((4, 4, 64), dtype=torch.bfloat16), torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="workspace"):
        tpa.qk_norm_rope_bwd(torch.zeros(4, dtype=torch.int32), q, k, q, k, torch.zeros((8, 64)), torch.ones(64), torch.ones(64),
                             workspace=ws)


def test_numbers_past_32_bits_are_not_cut(tpa, call):
    for window in (-1, -2 ** 32 + 5, -2 ** 63):
        with pytest.raises(ValueError, match="window"):
            tpa.paged_attn_fwd(**call, window=window)
    for most in (2 ** 31, 2 ** 32 + 1, -2 ** 32 + 1):
        with pytest.raises(ValueError, match="max_q_len"):
            tpa.paged_attn_fwd(**{**call, "max_q_len": most})
        with pytest.raises(ValueError, match="max_q_len"):
            tpa.paged_attn_workspace_bytes(most, 4, 2, 64)
    with pytest.raises(ValueError, match="n_positions"):
        tpa.rope_table(2 ** 32 + 1, 16, device="meta")
    long = torch.zeros((1, 1, 1)).expand(2 ** 32 + 1, 1, 1)  # as many sequences, of one probability each
    with pytest.raises(ValueError, match="sequences"):
        tpa.verify_drafts(long, torch.zeros((1, 0), dtype=torch.int32).expand(2 ** 32 + 1, 0),
                          torch.zeros((1, 0)).expand(2 ** 32 + 1, 0), torch.zeros(1).expand(2 ** 32 + 1))


def test_a_build_that_does_not_fit_has_its_own_status(tpa):
    from prefix_shared_tree_attention_gb300 import STATUS
    assert STATUS[-9] == "TPA_ERR_BAD_BUILD"
    f = tpa.lib().tpa_status_string
    f.restype = C.c_char_p
    assert f(-9) == b"TPA_ERR_BAD_BUILD"
