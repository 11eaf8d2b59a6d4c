"""GPU parity of the head norms and rotary positions (tpa_rope_table,
tpa_qk_norm_rope_fwd / _bwd) against fp64.

Tolerances.  An fp32 result is formed from a few products and sums: the norm's
sum of squares (16 fused products in a lane, 3 additions, halved by the root),
rsqrt, the products with it, the weight and the cosine or sine, and one
addition: fewer than 32 roundings of 2^-24 (rsqrt counted as 4), so it is
within 2^-19 of the magnitudes it was summed from.  A gradient takes the norm,
the mean of the products and two more products: within 2^-18.  A bf16 result
adds half a step, 2^-8 of the value.  A weight's gradient is a sum of n terms
that are within 2^-19 each, added in fp32: n 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from oracle.rope import norm_rope, norm_rope_grad, rope_angles
from synth import random_small_sequences
from _pipeline import check_guards, guarded, pack_and_upload

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
EPS = 1e-6


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _close(got, ref, size, rel, half, what):
    g, r = got.detach().double().cpu(), ref.cpu()
    assert g.shape == r.shape and torch.isfinite(g).all(), what
    off = (g - r).abs() - (rel * size.cpu() * (1 + half) + half * r.abs())
    assert off.max().item() <= 0 if off.numel() else True, f"{what}: {off.max().item():.3e} past the bound"


def _inputs(rows, hq, hkv, d, seed, fused=False, limit=500):
    g = torch.Generator().manual_seed(seed)
    if fused:
        qkv = torch.randn((rows, (hq + 2 * hkv) * d), generator=g).to(torch.bfloat16).cuda()
        q, k = qkv[:, :hq * d].view(rows, hq, d), qkv[:, hq * d:(hq + hkv) * d].view(rows, hkv, d)
    else:
        q = torch.randn((rows, hq, d), generator=g).to(torch.bfloat16).cuda()
        k = torch.randn((rows, hkv, d), generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(-1, limit, (rows,), generator=g, dtype=torch.int32)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    return q, k, pos, w


CASES = [  # rows, hq, hkv, d, rot, interleaved, weights, fused
    (1, 1, 1, 64, 64, False, "f32", False), (1, 32, 8, 128, 128, False, "f32", True),
    (7, 3, 1, 128, 128, True, "bf16", False), (33, 5, 5, 64, 32, False, "bf16", True),
    (100, 17, 1, 128, 64, True, None, True), (257, 9, 3, 128, 16, False, "f32", False),
    (64, 4, 4, 64, 16, True, None, False), (1025, 40, 8, 64, 48, False, "f32", True),
    (300, 33, 33, 128, 112, False, "f32", True), (1500, 16, 4, 128, 128, False, "f32", True),
    (2500, 12, 12, 64, 32, True, "bf16", False), (5000, 2, 1, 128, 128, False, "f32", True)]

# Calls of few bytes and of many take other kernels
SIZES = [(50, 4, 2, 64), (700, 16, 4, 128)]


def _weights(kind, w):
    return (None, None) if kind is None else tuple(x.to(torch.bfloat16) if kind == "bf16" else x for x in w)


@pytest.mark.parametrize("rows,hq,hkv,d,rot,inter,weights,fused", CASES)
def test_forward(tpa, rows, hq, hkv, d, rot, inter, weights, fused):
    q, k, pos, w = _inputs(rows, hq, hkv, d, rows + hq, fused)
    wq, wk = _weights(weights, w)
    table = tpa.rope_table(500, rot)
    bq, oq = guarded(q.shape, torch.bfloat16)
    bk, ok = guarded(k.shape, torch.bfloat16)
    tpa.qk_norm_rope_fwd(pos.cuda(), q, k, table, wq, wk, eps=EPS, interleaved=inter, out=(oq, ok))
    tpa.sync_status()
    check_guards(bq, "q")
    check_guards(bk, "k")
    row = table.cpu()[pos.clamp(min=0).long()]
    pad = (pos < 0)
    for x, wt, got in ((q, wq, oq), (k, wk, ok)):
        ref, size = norm_rope(x.cpu(), None if wt is None else wt.cpu(), row, EPS, inter)
        ref[pad] = 0
        size[pad] = 0
        _close(got, ref, size, 2.0 ** -19, HALF, "forward")
        assert (got.cpu()[pad] == 0).all()


@pytest.mark.parametrize("gin,gout", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,hq,hkv,d,rot,inter,weights,fused", CASES)
def test_gradient(tpa, rows, hq, hkv, d, rot, inter, weights, fused, gin, gout):
    t = {"f32": torch.float32, "bf16": torch.bfloat16}
    q, k, pos, w = _inputs(rows, hq, hkv, d, rows + hq, fused)
    wq, wk = _weights(weights, w)
    g = torch.Generator().manual_seed(9)
    gq, gk = (torch.randn(x.shape, generator=g).to(t[gin]).cuda() for x in (q, k))
    table = tpa.rope_table(500, rot)
    bq, oq = guarded(q.shape, t[gout])
    bk, ok = guarded(k.shape, t[gout])
    _, _, dwq, dwk = tpa.qk_norm_rope_bwd(pos.cuda(), gq, gk, q, k, table, wq, wk, eps=EPS, interleaved=inter,
                                          grad_dtype=t[gout], out=(oq, ok))
    tpa.sync_status()
    check_guards(bq, "dq")
    check_guards(bk, "dk")
    real = pos >= 0
    row = table.cpu()[pos[real].long()]
    for gr, x, wt, got, dw in ((gq, q, wq, oq, dwq), (gk, k, wk, ok, dwk)):
        dx, rdw, size, dsize = norm_rope_grad(gr.cpu()[real], x.cpu()[real], None if wt is None else wt.cpu(), row, EPS,
                                              inter)
        _close(got[real.cuda()], dx, size, 2.0 ** -18, HALF if gout == "bf16" else 0.0, "dx")
        assert (got.cpu()[~real] == 0).all()
        if wt is None:
            assert dw is None
        else:
            n = int(real.sum()) * x.shape[1] + 64
            _close(dw, rdw, dsize, 2.0 ** -19 + n * 2.0 ** -24, 0.0, "dw")


def test_gradient_against_differences(tpa):
    # the kernels' own forward, at steps that its bf16 outputs resolve: f(x + e u) - f(x - e u) = 2 e <dx, u> + O(e^3)
    rows, hq, hkv, d = 64, 4, 2, 128
    q, k, pos, (wq, wk) = _inputs(rows, hq, hkv, d, 5)
    pos = pos.clamp(min=0).cuda()
    table = tpa.rope_table(500, d)
    g = torch.Generator().manual_seed(11)
    gq = torch.randn(q.shape, generator=g).cuda()
    dq, _, dwq, _ = tpa.qk_norm_rope_bwd(pos, gq, torch.zeros(k.shape, device="cuda"), q, k, table, wq, wk,
                                         grad_dtype=torch.float32)

    def f(x, w):
        return (tpa.qk_norm_rope_fwd(pos, x, k, table, w, wk)[0].double() * gq).sum().item()

    u = torch.randn(q.shape, generator=g).cuda()
    up, down = (q + 0.05 * u).to(torch.bfloat16), (q - 0.05 * u).to(torch.bfloat16)
    step = up.double() - down.double()
    want = (dq.double() * step).sum().item()
    # each output is off by up to 2^-8 of itself: a random sum over them, 6 standard deviations of a uniform error
    noise = 6 * (gq.double() ** 2 * (2.0 ** -8 * 3) ** 2 / 3).sum().sqrt().item()
    assert abs(f(up, wq) - f(down, wq) - want) <= noise + 0.02 * (dq.double() * step).norm().item()
    v = torch.randn(d, generator=g).cuda()
    want = 2 * 0.1 * (dwq.double() * v).sum().item()
    assert abs(f(q, wq + 0.1 * v) - f(q, wq - 0.1 * v) - want) <= noise  # linear in w


def test_table(tpa):
    for rot, kw in ((64, {}), (128, dict(base=500000.0)), (16, dict(scale=0.7)),
                    (32, dict(inv_freq=[0.5 ** j for j in range(16)]))):
        n = 70001
        got = tpa.rope_table(n, rot, **kw).double().cpu()
        ref = rope_angles(n, rot, **kw)
        # the angle n f in fp64 is off by a rounding of f and one of the product; pow and sincos by a few 2^-53 more
        assert ((got - ref).abs() <= 2.0 ** -24 * ref.abs() + 8 * n * 2.0 ** -52).all()


@pytest.mark.parametrize("rows,hq,hkv,d", SIZES)
def test_padding_may_hold_anything(tpa, rows, hq, hkv, d):
    q, k, pos, (wq, wk) = _inputs(rows, hq, hkv, d, 3)
    pos[10:20] = -1
    clean = tpa.qk_norm_rope_fwd(pos.cuda(), q, k, (table := tpa.rope_table(500, 64)), wq, wk)
    g = [torch.randn(x.shape, device="cuda") for x in (q, k)]
    gclean = tpa.qk_norm_rope_bwd(pos.cuda(), *g, q, k, table, wq, wk, grad_dtype=torch.float32)
    for x in (q, k, *g):
        x[10:15] = float("nan")
        x[15:20] = float("inf")
    dirty = tpa.qk_norm_rope_fwd(pos.cuda(), q, k, table, wq, wk)
    gdirty = tpa.qk_norm_rope_bwd(pos.cuda(), *g, q, k, table, wq, wk, grad_dtype=torch.float32)
    tpa.sync_status()
    assert all(torch.equal(a, b) for a, b in zip((*clean, *gclean), (*dirty, *gdirty)))


@pytest.mark.parametrize("rows,heads", [(2, 1), (900, 20)])
def test_infinite_value_beside_the_rotation(tpa, rows, heads):
    # without a norm a value that is not turned passes as it is, its neighbours too
    q = torch.ones((rows, heads, 64), dtype=torch.bfloat16, device="cuda")
    q[:, :, 33] = float("inf")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") % 8
    table = tpa.rope_table(8, 32)
    got, _ = tpa.qk_norm_rope_fwd(pos, q, q.clone(), table)
    assert torch.equal(got[..., 32:], q[..., 32:])


@pytest.mark.parametrize("rows,hq,hkv,d", [(9, 4, 2, 64), (700, 16, 4, 128)])
def test_position_past_the_table(tpa, rows, hq, hkv, d):
    q, k, pos, (wq, wk) = _inputs(rows, hq, hkv, d, 4)
    pos = pos.clamp(min=0)
    table = tpa.rope_table(500, 64)
    want = tpa.qk_norm_rope_fwd(pos.cuda(), q, k, table, wq, wk)
    bad = pos.clone()
    bad[3], bad[5] = 500, 2 ** 31 - 1
    got = tpa.qk_norm_rope_fwd(bad.cuda(), q, k, table, wq, wk)
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()
    tpa.sync_status()
    keep = [i for i in range(rows) if i not in (3, 5)]
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep]) and (a[[3, 5]] == 0).all()
    got = tpa.qk_norm_rope_bwd(bad.cuda(), *want, q, k, table, wq, wk)
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()
    assert (got[0][[3, 5]] == 0).all() and all(torch.isfinite(x).all() for x in got)


@pytest.mark.parametrize("rows", [70, 1100])
def test_in_place_and_strided_outputs(tpa, rows):
    q, k, pos, (wq, wk) = _inputs(rows, 8, 2, 128, 6, fused=True)
    pos, table = pos.cuda(), tpa.rope_table(500, 128)
    want = tpa.qk_norm_rope_fwd(pos, q, k, table, wq, wk)
    fresh = torch.zeros((rows, 12 * 128), dtype=torch.bfloat16, device="cuda")
    views = fresh[:, :1024].view(rows, 8, 128), fresh[:, 1024:1280].view(rows, 2, 128)
    tpa.qk_norm_rope_fwd(pos, q, k, table, wq, wk, out=views)
    assert all(torch.equal(a, b) for a, b in zip(views, want)) and (fresh[:, 1280:] == 0).all()
    gw = tpa.qk_norm_rope_bwd(pos, *want, q, k, table, wq, wk)
    g = [x.clone() for x in want]
    tpa.qk_norm_rope_bwd(pos, *g, q, k, table, wq, wk, out=tuple(g))
    assert torch.equal(g[0], gw[0]) and torch.equal(g[1], gw[1])
    tpa.qk_norm_rope_fwd(pos, q, k, table, wq, wk, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("hq,hkv", [(2, 1), (400, 20)])
def test_rows_far_apart(tpa, hq, hkv):
    # byte offsets past 2^32: 5 GB between the first row and the last
    rows, stride = 40, 1 << 26
    flat = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda")
    q = flat.as_strided((rows, hq, 64), (stride, 64, 1))
    k = flat[64 * hq:].as_strided((rows, hkv, 64), (stride, 64, 1))
    src, ksrc, pos, (wq, wk) = _inputs(rows, hq, hkv, 64, 8)
    q.copy_(src)
    k.copy_(ksrc)
    table = tpa.rope_table(500, 64)
    want = tpa.qk_norm_rope_fwd(pos.cuda(), src, ksrc, table, wq, wk)
    got = tpa.qk_norm_rope_fwd(pos.cuda(), q, k, table, wq, wk, out=(q, k))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("hq,hkv,d,norm", [(32, 8, 128, True), (12, 6, 64, False)])
def test_the_same_in_one_call_and_in_many(tpa, hq, hkv, d, norm):
    q, k, pos, (wq, wk) = _inputs(1300, hq, hkv, d, 12, fused=True)
    pos, table = pos.cuda(), tpa.rope_table(500, d)
    w = (wq, wk) if norm else (None, None)
    want = tpa.qk_norm_rope_fwd(pos, q, k, table, *w)
    parts = [tpa.qk_norm_rope_fwd(pos[i:i + 37], q[i:i + 37], k[i:i + 37], table, *w) for i in range(0, 1300, 37)]
    assert all(torch.equal(torch.cat(x), y) for x, y in zip(zip(*parts), want))
    tpa.sync_status()


def test_no_rows(tpa):
    q, k, pos, (wq, wk) = _inputs(0, 4, 2, 64, 3)
    table = tpa.rope_table(8, 64)
    a, b = tpa.qk_norm_rope_fwd(pos.cuda(), q, k, table, wq, wk)
    dq, dk, dwq, dwk = tpa.qk_norm_rope_bwd(pos.cuda(), q, k, q, k, table, wq, wk)
    tpa.sync_status()
    assert a.shape == q.shape and dk.shape == k.shape and (dwq == 0).all() and (dwk == 0).all()


def test_same_results_twice_on_a_stream_and_from_a_graph(tpa):
    q, k, pos, (wq, wk) = _inputs(2000, 16, 2, 128, 10)
    pos, table = pos.cuda(), tpa.rope_table(500, 128)

    def both():
        y = tpa.qk_norm_rope_fwd(pos, q, k, table, wq, wk)
        return *y, *tpa.qk_norm_rope_bwd(pos, *y, q, k, table, wq, wk, grad_dtype=torch.float32)

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    q.copy_(torch.randn_like(q))
    want = both()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, kept))


def test_on_a_packed_tree_with_the_attention(tpa):
    """norm + rotation -> tree attention -> its gradients -> gradients of the projections, against autograd in fp64."""
    rng = np.random.default_rng(21)
    seqs = random_small_sequences(rng, 12, 150, 3, min_len=2)
    T = 256
    tree, dtree, mask = pack_and_upload(tpa, seqs, T)
    B, Hq, Hkv, d = tree.n_trees, 4, 2, 64
    arr = tree.arrays()
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn((B, T, (Hq + 2 * Hkv) * d), generator=g).to(torch.bfloat16).cuda()
    q = qkv[..., :Hq * d].view(B, T, Hq, d)
    k = qkv[..., Hq * d:(Hq + Hkv) * d].view(B, T, Hkv, d)
    v = qkv[..., (Hq + Hkv) * d:].reshape(B, T, Hkv, d).contiguous()
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    do = torch.randn((B, T, Hq, d), generator=g).to(torch.bfloat16).cuda()
    pad = torch.from_numpy(np.arange(T)[None] >= arr["n_tokens"][:, None]).cuda()
    q[pad] = float("nan")  # a projection's padding rows may hold anything
    k[pad] = float("nan")
    table = tpa.rope_table(T, d)
    y = tpa.qk_norm_rope_fwd(dtree, q, k, table, wq, wk)
    depth = torch.from_numpy(arr["depth"]).cuda()
    alone = tpa.qk_norm_rope_fwd(torch.where(pad, -1, depth).to(torch.int32), q, k, table, wq, wk)
    assert all(torch.equal(a, b) for a, b in zip(y, alone)) and (y[0][pad] == 0).all() and (y[1][pad] == 0).all()
    o, lse = tpa.tree_attn_fwd(dtree, mask, *y, v)
    gq, gk, _ = tpa.tree_attn_bwd(dtree, mask, *y, v, o, lse, do)
    dq, dk, dwq, dwk = tpa.qk_norm_rope_bwd(dtree, gq, gk, q, k, table, wq, wk, grad_dtype=torch.float32)
    tpa.sync_status()

    ends = torch.from_numpy(arr["subtree_end"]).cuda()
    i = torch.arange(T, device="cuda")
    sees = (i[None, :, None] >= i[None, None]) & (i[None, :, None] <= ends[:, None]) & ~pad[:, :, None]
    q64, k64 = (torch.where(pad[..., None, None], 0.0, x.double()).requires_grad_() for x in (q, k))
    w64 = [w.double().requires_grad_() for w in (wq, wk)]
    row = table.double()[depth.long()]
    c, s = (x[:, :, None].detach() for x in (row[..., :d // 2], row[..., d // 2:]))

    def rope(x, w):
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    qr, kr = rope(q64, w64[0]), rope(k64, w64[1]).repeat_interleave(Hq // Hkv, 2)
    x = torch.einsum("bihd,bjhd->bhij", qr, kr) / d ** 0.5
    p = torch.softmax(x.masked_fill(~sees[:, None], -1e30), -1) * sees[:, None]
    out = torch.einsum("bhij,bjhd->bihd", p, v.double().repeat_interleave(Hq // Hkv, 2))
    grads = torch.autograd.grad((out * do.double()).sum(), (q64, k64, *w64))
    # the bounds of the attention's own gradients (2e-2, 5e-3), doubled for the bf16 roundings of q, k between the two
    # operators; a weight's gradient adds up the errors of all rows
    for name, got, ref in zip(("dq", "dk", "dwq", "dwk"), (dq, dk, dwq, dwk), grads):
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        assert torch.isfinite(got).all() and rel <= 1e-2, f"{name}: rel-L2 {rel:.3e}"
