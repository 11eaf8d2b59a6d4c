"""Refusals of the policy's operators (CPU): every call that its description
does not allow comes back as an error before anything is launched."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    return tpa


P = 4096  # an aligned address that no refused call follows
BAD = -1


def _rope(**kw):
    from prefix_shared_tree_attention_gb300._abi import RopeParams
    r = RopeParams()
    r.table, r.table_rows, r.rot_dim, r.eps = P, 100, 64, 1e-6
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _fwd(L, rope=None, positions=P, n_tokens=None, t_pad=0, rows=4, q=P, sq=256, k=P, sk=128, qo=P, so=256, ko=P,
         sko=128, hq=4, hkv=2, d=64):
    return L.tpa_qk_norm_rope_fwd(positions, n_tokens, t_pad, rows, q, sq, k, sk, C.byref(rope or _rope()), qo, so, ko,
                                  sko, hq, hkv, d, None)


@pytest.mark.parametrize("kw", [
    dict(d=96), dict(hq=0), dict(hkv=0), dict(rows=-1), dict(positions=None), dict(q=None), dict(k=None),
    dict(qo=None), dict(ko=None), dict(q=P + 2), dict(sq=255), dict(sq=260), dict(so=100), dict(sk=127),
    dict(rows=1 << 31), dict(n_tokens=P, t_pad=0), dict(n_tokens=P, t_pad=3), dict(sq=1 << 40)])
def test_norm_rope_refusals(tpa, kw):
    assert _fwd(tpa.lib(), **kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(table=P + 4), dict(rot_dim=24), dict(rot_dim=0), dict(rot_dim=80), dict(table_rows=0),
    dict(q_weight=P), dict(k_weight=P), dict(q_weight=P, k_weight=P + 2), dict(weight_type=7), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf"))])
def test_rope_parameter_refusals(tpa, kw):
    assert _fwd(tpa.lib(), rope=_rope(**kw)) == BAD


def test_no_rows_is_no_work(tpa):
    assert _fwd(tpa.lib(), rows=0) == 0


def _bwd(L, rope=None, gin=0, gout=1, dwq=P, dwk=P, ws=P, nbytes=1 << 24, q=P, k=P, dq=P, sdq=256, rows=4, gq=P,
         sgq=256, d=64):
    return L.tpa_qk_norm_rope_bwd(P, None, 0, rows, gq, sgq, P, 128, gin, q, 256, k, 128,
                                  C.byref(rope or _rope(q_weight=P, k_weight=P)), dq, sdq, P, 128, gout, dwq, dwk, ws,
                                  nbytes, 4, 2, d, None)


@pytest.mark.parametrize("kw,status", [
    (dict(gin=2), BAD), (dict(gout=-1), BAD), (dict(dwq=None), BAD), (dict(dwk=P + 2), BAD), (dict(ws=None), BAD),
    (dict(ws=P + 8), BAD), (dict(nbytes=1000), -8), (dict(q=None), BAD), (dict(k=None), BAD), (dict(dq=None), BAD),
    (dict(sdq=250), BAD), (dict(gq=P + 8), BAD), (dict(sgq=258, gin=0), BAD), (dict(d=32), BAD), (dict(rows=-4), BAD)])
def test_norm_rope_grad_refusals(tpa, kw, status):
    assert _bwd(tpa.lib(), **kw) == status


def test_grad_workspace_bytes(tpa):
    f = tpa.lib().tpa_qk_norm_rope_bwd_workspace_bytes
    assert f(64) > 0 and f(128) == 2 * f(64) and f(96) == 0 and f(0) == 0


@pytest.mark.parametrize("kw", [dict(table=None), dict(table=P + 4), dict(n=0), dict(rot=8), dict(rot=144),
                                dict(rot=24), dict(base=0.0), dict(base=-1.0), dict(base=float("nan")),
                                dict(scale=float("inf")), dict(freq=float("nan"))])
def test_rope_table_refusals(tpa, kw):
    a = dict(table=P, n=10, rot=32, base=1e4, scale=1.0, freq=None)
    a.update(kw)
    fr = None if a["freq"] is None else (C.c_double * 16)(*[a["freq"]] * 16)
    assert tpa.lib().tpa_rope_table(a["table"], a["n"], a["rot"], a["base"], fr, a["scale"], None) == BAD


def _paged(**kw):
    from prefix_shared_tree_attention_gb300._abi import PagedView
    v = PagedView()
    v.k_cache = v.v_cache = v.pages = v.offsets = v.kv_lens = P
    v.n_pages, v.page_size, v.n_seqs, v.max_pages, v.page_stride = 10, 16, 2, 4, 4
    v.n_heads_kv, v.head_dim, v.n_rows = 2, 64, 3
    for k, x in kw.items():
        setattr(v, k, x)
    return v


BAD_PAGED = [
    dict(k_cache=None), dict(v_cache=None), dict(pages=None), dict(offsets=None), dict(kv_lens=None),
    dict(k_cache=P + 8), dict(v_cache=P + 2), dict(head_dim=80), dict(page_size=8), dict(page_size=48),
    dict(page_size=256), dict(n_pages=0), dict(n_seqs=0), dict(max_pages=0), dict(page_stride=3), dict(n_rows=-1), dict(n_rows=1 << 30),
    dict(n_heads_kv=0), dict(n_pages=1 << 27, n_heads_kv=1), dict(max_pages=1 << 27, page_stride=1 << 27)]


def _append(L, view, k=P, sk=128, v=P, sv=128, q=None, sq=0, qo=None, so=0, hq=0, rope=None):
    return L.tpa_paged_append(C.byref(view), k, sk, v, sv, q, sq, qo, so, hq, C.byref(rope or _rope()), None)


@pytest.mark.parametrize("kw", BAD_PAGED)
def test_paged_view_refusals(tpa, kw):
    assert _append(tpa.lib(), _paged(**kw)) == BAD


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=P + 4), dict(sk=64), dict(sv=132), dict(hq=-1),
                                dict(hq=4), dict(hq=4, q=P, sq=256), dict(hq=4, q=P, sq=200, qo=P, so=256)])
def test_append_refusals(tpa, kw):
    assert _append(tpa.lib(), _paged(), **kw) == BAD


def test_append_of_nothing(tpa):
    assert _append(tpa.lib(), _paged(n_rows=0)) == 0


def _attend(L, view, q=P, sq=256, o=P, lse=P, hq=4, max_q=5, scale=0.0, window=0, ws=P, nbytes=1 << 30):
    return L.tpa_paged_attn_fwd(C.byref(view), q, sq, o, lse, hq, max_q, scale, window, ws, nbytes, None)


@pytest.mark.parametrize("kw", BAD_PAGED)
def test_attend_view_refusals(tpa, kw):
    assert _attend(tpa.lib(), _paged(**kw)) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), BAD), (dict(o=None), BAD), (dict(lse=None), BAD), (dict(ws=None), BAD), (dict(q=P + 8), BAD),
    (dict(o=P + 4), BAD), (dict(lse=P + 2), BAD), (dict(ws=P + 128), BAD), (dict(sq=128), BAD), (dict(sq=257), BAD),
    (dict(hq=3), BAD), (dict(hq=0), BAD), (dict(max_q=0), BAD), (dict(window=-1), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(nbytes=1000), -8)])
def test_attend_refusals(tpa, kw, status):
    assert _attend(tpa.lib(), _paged(), **kw) == status


def test_attend_of_nothing(tpa):
    assert _attend(tpa.lib(), _paged(n_rows=0)) == 0


def test_attend_workspace_bytes(tpa):
    f = tpa.paged_attn_workspace_bytes
    assert 0 < f(1, 32, 8, 64) < f(1, 32, 8, 128) and f(1, 32, 8, 128) <= f(5, 32, 8, 128)
    assert f(0, 8, 8, 128) == f(1, 6, 4, 128) == f(1, 8, 8, 96) == f(1, 0, 8, 64) == 0


def _verify(L, target=P, ts=300, draft=None, ds=0, toks=P, nd=None, ua=P, un=P, out=P, acc=P, S=2, K=2, V=100):
    return L.tpa_verify_drafts(target, ts, draft, ds, toks, nd, ua, un, out, acc, S, K, V, None)


@pytest.mark.parametrize("kw", [dict(target=None), dict(toks=None), dict(ua=None), dict(un=None), dict(out=None),
                                dict(acc=None), dict(ts=299), dict(draft=P, ds=199), dict(S=-1), dict(K=-1),
                                dict(K=1025, ts=1 << 20), dict(V=0), dict(V=(1 << 30) + 1, ts=1 << 33),
                                dict(target=P + 2), dict(nd=P + 1)])
def test_verify_refusals(tpa, kw):
    assert _verify(tpa.lib(), **kw) == BAD


def test_verify_of_no_sequence(tpa):
    assert _verify(tpa.lib(), S=0) == 0


def test_python_refusals(tpa):
    bf = torch.bfloat16
    q, k = torch.zeros((4, 4, 64), dtype=bf), torch.zeros((4, 2, 64), dtype=bf)
    pos, table = torch.zeros(4, dtype=torch.int32), torch.zeros((8, 64))
    for bad in (dict(q=q.float()), dict(q=q[:, :, ::2]), dict(q=q.transpose(0, 1)), dict(k=k[:3]),
                dict(positions=pos.long()), dict(positions=pos[:3]), dict(table=table.double()),
                dict(q_weight=torch.ones(64)), dict(q_weight=torch.ones(64), k_weight=torch.ones(32)), dict()):
        a = dict(positions=pos, q=q, k=k, table=table)
        a.update(bad)
        with pytest.raises(ValueError):  # the last: tensors of the host
            tpa.qk_norm_rope_fwd(**a)
    with pytest.raises(ValueError):
        tpa.qk_norm_rope_bwd(pos, q, k.float(), q, k, table)
    with pytest.raises(ValueError):
        tpa.qk_norm_rope_bwd(pos, q, k, None, None, table, torch.ones(64), torch.ones(64))
    cache = torch.zeros((3, 2, 16, 64), dtype=bf)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(k_cache=cache, v_cache=cache.clone(), pages=i32(2, 3), offsets=i32(3), kv_lens=i32(2), k=k, v=k.clone())
    for bad in (dict(k_cache=cache.float()), dict(v_cache=cache[:2]), dict(pages=i32(2, 3).long()), dict(offsets=i32(2)),
                dict(kv_lens=i32(3)), dict(v=k[:2]), dict(q=q[:3]), dict(q_out=q), dict(k=k[:, :1], v=k[:, :1]), dict()):
        with pytest.raises(ValueError):
            tpa.paged_append(**{**good, **bad})
    good = {x: good[x] for x in ("k_cache", "v_cache", "pages", "offsets", "kv_lens")} | dict(q=q, max_q_len=2)
    for bad in (dict(q=q[None]), dict(q=q.float()), dict(out=q.float()), dict(out=q[:3]), dict(lse=torch.zeros(4)),
                dict(lse=torch.zeros((4, 4), dtype=torch.float64)), dict(pages=i32(2, 3)[:, ::2]), dict()):
        with pytest.raises(ValueError):
            tpa.paged_attn_fwd(**{**good, **bad})
    p, x, u, n = torch.zeros((2, 3, 10)), i32(2, 2), torch.zeros((2, 2)), torch.zeros(2)
    for bad in (dict(target_probs=p.double()), dict(target_probs=p[:, :, ::2]), dict(draft_tokens=x.long()),
                dict(u_accept=u[:, :1]), dict(u_next=u), dict(draft_probs=p), dict(n_drafts=i32(3)), dict()):
        with pytest.raises(ValueError):
            tpa.verify_drafts(**{**dict(target_probs=p, draft_tokens=x, u_accept=u, u_next=n), **bad})
    with pytest.raises(ValueError):
        tpa.rope_table(10, 32, inv_freq=[1.0], device="cpu")
    with pytest.raises(ValueError):
        tpa.rope_table(10, 32, device="cpu")
