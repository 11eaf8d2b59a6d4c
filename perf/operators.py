"""Operators of the policy model around tree attention, as cases to measure.

A policy is trained on packed trees and sampled from a paged cache.  Four
operators stand between its projections and the two attentions:

- ``norm_rope`` / ``norm_rope_grad``: RMS norm of every query and key head and
  the rotation by position, one pass, and its gradient (training);
- ``append``: the same on the new tokens of a batch of sequences, with the keys
  and values written into pages of a cache (sampling);
- ``attend``: attention of each sequence's new tokens over its pages;
- ``verify``: drafted tokens accepted or rejected against the policy's
  probabilities, and the next token drawn, from given uniform numbers.

``run`` computes them by elementary torch operations, or through the package
where ``own`` is true.  ``exact`` gives the same outputs in 64 bits, written
apart from both.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------ the cases

def _rope(name, grad, n, real, hq, hkv, d, rot, interleaved, norm, grad_type):
    return {"name": name, "kind": "norm_rope_grad" if grad else "norm_rope", "n": n, "real": real, "hq": hq,
            "hkv": hkv, "d": d, "rot": rot, "interleaved": interleaved, "norm": norm, "grad_type": grad_type}


def _append(name, seqs, q_low, q_high, kv_low, kv_high, hq, hkv, d, page, norm):
    return {"name": name, "kind": "append", "seqs": seqs, "q_low": q_low, "q_high": q_high, "kv_low": kv_low,
            "kv_high": kv_high, "hq": hq, "hkv": hkv, "d": d, "page": page, "norm": norm, "share": 1, "prefix": 0}


def _attend(name, seqs, q_low, q_high, kv_low, kv_high, hq, hkv, d, page, window, share, prefix):
    return {"name": name, "kind": "attend", "seqs": seqs, "q_low": q_low, "q_high": q_high, "kv_low": kv_low,
            "kv_high": kv_high, "hq": hq, "hkv": hkv, "d": d, "page": page, "window": window, "share": share,
            "prefix": prefix}


def _verify(name, seqs, drafts, vocab, draft_probs):
    return {"name": name, "kind": "verify", "seqs": seqs, "drafts": drafts, "vocab": vocab,
            "draft_probs": draft_probs}


def listed():
    return [
        # the tiny workload's tree: one micro-batch of 1024 positions, 821 of them tokens
        _rope("norm_rope tiny tree", False, 1024, 821, 4, 4, 64, 64, False, True, "bf16"),
        # the few-shot workload: one tree of 65536 positions
        _rope("norm_rope few-shot tree", False, 65536, 56311, 32, 8, 128, 128, False, True, "bf16"),
        # a GRPO step's three trees of 8192 positions, gradients in bf16
        _rope("norm_rope grad GRPO trees", True, 24576, 23999, 32, 8, 128, 128, False, True, "bf16"),
        # the agentic tree, attention gradients in fp32, half of each head rotated
        _rope("norm_rope grad agentic", True, 32768, 16701, 16, 2, 128, 64, True, True, "f32"),
        # one decode step of 64 samples: a token each
        _append("append decode step", 64, 1, 1, 300, 3000, 32, 8, 128, 16, True),
        # the prompts of a batch, 256 to 1024 tokens each
        _append("append prompts", 32, 256, 1024, 256, 1024, 16, 2, 128, 64, True),
        # a decode step of 8 prompts x 8 samples that share their prompt's pages
        _attend("attend decode GRPO", 64, 1, 1, 300, 3000, 32, 8, 128, 16, 0, 8, 256),
        # one long agentic trajectory, one token: the work has to be split along the keys
        _attend("attend decode long", 1, 1, 1, 130001, 130001, 16, 2, 128, 64, 0, 1, 0),
        # five drafted tokens of each of 16 sequences
        _attend("attend drafts", 16, 5, 5, 1000, 8000, 32, 8, 128, 32, 0, 1, 0),
        # a chunk of a prompt behind what is cached already
        _attend("attend prefill chunk", 1, 4001, 4001, 32003, 32003, 32, 8, 128, 64, 0, 1, 0),
        # one sequence's drafts, the tokenised workloads' ids
        _verify("verify one", 1, 4, 32000, True),
        # a batch of drafts at the logits workload's vocabulary
        _verify("verify batch", 64, 5, 151936, True),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["norm_rope", "norm_rope_grad", "append", "attend", "attend", "verify"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    if kind in ("norm_rope", "norm_rope_grad"):
        n = _log(rng, 1, 32768)
        rot = rng.choice([d, d, d // 2, 16])
        c = _rope("", kind == "norm_rope_grad", n, rng.randint(0, n), hq, hkv, d, rot, rng.random() < 0.3,
                  rng.random() < 0.8, rng.choice(["bf16", "f32"]))
    elif kind == "append":
        seqs = _log(rng, 1, 96)
        high = _log(rng, 1, max(1, 16384 // seqs))
        low = rng.randint(1, high)
        c = _append("", seqs, low, high, high, high + _log(rng, 1, 2000), hq, hkv, d, page, rng.random() < 0.7)
    elif kind == "attend":
        window = rng.choice([0, 0, 0, 100, 1000])
        form = rng.choice(["decode", "drafts", "chunk"])
        if form == "decode":
            seqs = _log(rng, 1, 96)
            kv = _log(rng, 1, max(2, 200000 // seqs))
            c = _attend("", seqs, 1, 1, rng.randint(1, kv), kv, hq, hkv, d, page, window, 1, 0)
        elif form == "drafts":
            seqs = _log(rng, 1, 48)
            kv = _log(rng, 10, max(20, 150000 // seqs))
            high = rng.randint(2, 9)
            c = _attend("", seqs, 1, high, rng.randint(high, max(high, kv)), max(high, kv), hq, hkv, d, page, window,
                        1, 0)
        else:
            seqs = _log(rng, 1, 8)
            high = _log(rng, 17, max(17, 3000 // seqs))
            kv = high + _log(rng, 1, max(2, 24000 // seqs))
            c = _attend("", seqs, rng.randint(1, high), high, rng.randint(high, kv), kv, hq, hkv, d, page, window,
                        1, 0)
    else:
        c = _verify("", _log(rng, 1, 64), rng.randint(1, 8), _log(rng, 1000, 151936), rng.random() < 0.7)
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs

def _lens(case):
    """New tokens and cached tokens (the new ones among them) of each sequence: the case's own, whatever the seed."""
    r = random.Random(1)
    q = [r.randint(case["q_low"], case["q_high"]) for _ in range(case["seqs"])]
    kv = [max(a, r.randint(case["kv_low"], case["kv_high"])) for a in q]
    return q, kv


def _pages(case):
    """The pages of each sequence, in order of use: shared ones for a group's prefix; and how many there are."""
    _, kv = _lens(case)
    p, rows, count = case["page"], [], 0
    for s, n in enumerate(kv):
        if s % case["share"] == 0:
            group = list(range(count, count + case["prefix"] // p))
            count += len(group)
        need = max(0, -(-n // p) - len(group))
        rows.append((group + list(range(count, count + need)))[:-(-n // p)])
        count += need
    return rows, count


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _table(positions, rot):
    """cos | sin of position x frequency, formed in 64 bits and rounded once: what a program keeps for its model."""
    freq = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kind = case["kind"]
    s = dict(case)
    if kind == "verify":
        n, k, v = case["seqs"], case["drafts"], case["vocab"]
        logits = 3 * _normal(g, n, k + 1, v)
        s["target"] = torch.softmax(logits, -1)
        # the draft model is close to the policy: most of its tokens are accepted
        draft = torch.softmax(logits[:, :k] + 0.5 * _normal(g, n, k, v), -1)
        pick = torch.multinomial(draft.view(n * k, v), 1, generator=g).view(n, k)
        s["tokens"] = pick.to(torch.int32)
        s["draft"] = draft if case["draft_probs"] else None
        s["n_drafts"] = torch.randint(0, k + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
        s["n_drafts"][0] = k
        s["u_accept"], s["u_next"] = _uniform(g, n, k), _uniform(g, n)
        return s
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case.get("norm"):
        s["wq"], s["wk"] = (1 + 0.2 * _normal(g, d) for _ in range(2))
    else:
        s["wq"] = s["wk"] = None
    if kind in ("norm_rope", "norm_rope_grad"):
        n = case["n"]
        # q and k are slices of the fused projection's rows, as a model has them
        qkv = _normal(g, n, (hq + 2 * hkv) * d).to(torch.bfloat16)
        s["q"] = qkv[:, :hq * d].view(n, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        # depths in a packed tree: runs that start again at branch points; padding behind the tokens
        i = torch.arange(n, device="cuda", dtype=torch.int32)
        s["positions"] = torch.where(i < case["real"], torch.where(i < 2048, i, 1024 + (i % 6143)), -1).to(torch.int32)
        s["table"] = _table(8192, case["rot"])
        if kind == "norm_rope_grad":
            t = torch.bfloat16 if case["grad_type"] == "bf16" else torch.float32
            s["type"] = t
            s["gq"], s["gk"] = _normal(g, n, hq, d).to(t), _normal(g, n, hkv, d).to(t)
        return s
    q_lens, kv_lens = _lens(case)
    rows, count = _pages(case)
    n, p = sum(q_lens), case["page"]
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    width = max(len(r) for r in rows)
    at = torch.tensor([r + [0] * (width - len(r)) for r in rows], device="cuda")
    s["pages"] = order[at].contiguous()
    s["offsets"] = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32, device="cuda")
    s["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    s["max_q"], s["max_kv"] = max(q_lens), max(kv_lens)
    s["k_cache"], s["v_cache"] = (_normal(g, count, hkv, p, d).to(torch.bfloat16) for _ in range(2))
    if kind == "append":
        qkv = _normal(g, n, (hq + 2 * hkv) * d).to(torch.bfloat16)
        s["q"] = qkv[:, :hq * d].view(n, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(n, hkv, d)
        s["table"] = _table(max(kv_lens), d)
    else:
        s["q"] = _normal(g, n, hq, d).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ the operators

def _normed(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _halves(x, rot, interleaved):
    r = x[..., :rot]
    return (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])


def _joined(a, b, rest, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _rotated(x, row, interleaved, back=False):
    """x [n, h, d] turned by the angles whose cos | sin are row [n, rot]; `back`: the other way."""
    rot = row.shape[1]
    c, s = row[:, None, :rot // 2], row[:, None, rot // 2:]
    s = -s if back else s
    a, b = _halves(x, rot, interleaved)
    return _joined(a * c - b * s, b * c + a * s, x[..., rot:], interleaved)


def _norm_rope(s, x, w):
    ok = (s["positions"] >= 0)[:, None, None]
    y = _rotated(_normed(x.float(), w), s["table"][s["positions"].clamp(min=0).long()], s["interleaved"])
    return torch.where(ok, y, 0.0).to(torch.bfloat16)


def _norm_rope_grad(s, g, x, w):
    ok = (s["positions"] >= 0)[:, None, None]
    z = _rotated(g.float(), s["table"][s["positions"].clamp(min=0).long()], s["interleaved"], back=True)
    z = torch.where(ok, z, 0.0)
    if w is None:
        return z.to(s["type"]), None
    x = torch.where(ok, x.float(), 0.0)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    h = x * r
    dw = (z * h).sum((0, 1))
    z = z * w
    return (r * (z - h * (z * h).mean(-1, keepdim=True))).to(s["type"]), dw


def _token_places(s, n):
    """For each new token: its sequence, its number among the sequence's new tokens, its position."""
    i = torch.arange(n, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"][1:], i, right=True)
    local = i - s["offsets"][seq]
    return seq, local.long(), (s["kv_lens"][seq] - (s["offsets"][seq + 1] - s["offsets"][seq]) + local).long()


def _append_plain(s):
    n, p = s["k"].shape[0], s["page"]
    seq, _, pos = _token_places(s, n)
    row = s["table"][pos]
    q = _rotated(_normed(s["q"].float(), s["wq"]), row, False).to(torch.bfloat16)
    k = _rotated(_normed(s["k"].float(), s["wk"]), row, False).to(torch.bfloat16)
    page, slot = s["pages"][seq, pos // p].long(), pos % p
    s["k_cache"][page, :, slot] = k
    s["v_cache"][page, :, slot] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _attend_plain(s):
    n, hq, d = s["q"].shape
    hkv, nseq, lq, lk = s["hkv"], s["seqs"], s["max_q"], s["max_kv"]
    g = hq // hkv
    seq, local, _ = _token_places(s, n)

    def keys(cache):
        c = cache[s["pages"].long()]                                # [seqs, pages, hkv, page, d]
        return c.transpose(1, 2).reshape(nseq, hkv, -1, d)[:, :, :lk].float()

    at = (s["offsets"][:-1, None] + torch.arange(lq, device="cuda")).clamp(max=n - 1).long()
    q = s["q"][at].view(nseq, lq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(nseq, hkv, g * lq, d).float()
    x = (q @ keys(s["k_cache"]).transpose(2, 3)).mul_(1 / math.sqrt(d)).view(nseq, hkv, g, lq, lk)
    q_len = (s["offsets"][1:] - s["offsets"][:-1])[:, None, None]
    pos = s["kv_lens"][:, None, None] - q_len + torch.arange(lq, device="cuda")[:, None]
    j = torch.arange(lk, device="cuda")
    seen = (j <= pos) & (j < s["kv_lens"][:, None, None])
    if s["window"]:
        seen = seen & (j > pos - s["window"])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(nseq, hkv, g * lq, lk) @ keys(s["v_cache"])).view(nseq, hkv, g, lq, d) / total.clamp(min=1e-30)
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(nseq, lq, hq, d)[seq, local]
    lse = lse.permute(0, 3, 1, 2).reshape(nseq, lq, hq)[seq, local]
    return o.to(torch.bfloat16), lse


def _verify_plain(s):
    p, x, n_drafts = s["target"], s["tokens"].long(), s["n_drafts"]
    n, k = x.shape
    i = torch.arange(k, device="cuda")
    rows = torch.arange(n, device="cuda")
    p_at = p[:, :k].gather(2, x[..., None])[..., 0].double()
    q_at = torch.ones_like(p_at) if s["draft"] is None else s["draft"].gather(2, x[..., None])[..., 0].double()
    fine = (s["u_accept"].double() * q_at < p_at) & (i < n_drafts[:, None])
    count = fine.int().cumprod(1).sum(1)
    turned_down = count < n_drafts
    last = count.clamp(max=k - 1)
    here = p[rows, count].double()
    if s["draft"] is None:
        other = torch.zeros_like(here).scatter_(1, x[rows, last][:, None], math.inf)
    else:
        other = s["draft"][rows, last].double()
    left = torch.where(turned_down[:, None], (here - other).clamp(min=0), here)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, here)
    sums = left.cumsum(1)
    picked = (sums <= s["u_next"].double()[:, None] * sums[:, -1:]).sum(1)
    picked = torch.minimum(picked, (left > 0).int().mul(torch.arange(1, left.shape[1] + 1, device="cuda")).amax(1) - 1)
    m = torch.arange(k + 1, device="cuda")
    out = torch.where(m < count[:, None], torch.nn.functional.pad(x, (0, 1)), -1)
    out = torch.where(m == count[:, None], picked[:, None], out)
    return out.to(torch.int32), count.to(torch.int32)


def _run_own(s):
    import prefix_shared_tree_attention_gb300 as tpa
    kind = s["kind"]
    if kind == "norm_rope":
        return tpa.qk_norm_rope_fwd(s["positions"], s["q"], s["k"], s["table"], s["wq"], s["wk"], eps=EPS,
                                    interleaved=s["interleaved"])
    if kind == "norm_rope_grad":
        return tpa.qk_norm_rope_bwd(s["positions"], s["gq"], s["gk"], s["q"], s["k"], s["table"], s["wq"], s["wk"],
                                    eps=EPS, interleaved=s["interleaved"], grad_dtype=s["type"])
    if kind == "append":
        q = tpa.paged_append(s["k_cache"], s["v_cache"], s["pages"], s["offsets"], s["kv_lens"], s["k"], s["v"],
                             q=s["q"], table=s["table"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS)
        return q, s["k_cache"], s["v_cache"]
    if kind == "attend":
        return tpa.paged_attn_fwd(s["k_cache"], s["v_cache"], s["pages"], s["offsets"], s["kv_lens"], s["q"],
                                  max_q_len=s["max_q"], window=s["window"])
    return tpa.verify_drafts(s["target"], s["tokens"], s["u_accept"], s["u_next"], draft_probs=s["draft"],
                             n_drafts=s["n_drafts"])


def run(state):
    if own:
        return _run_own(state)
    s, kind = state, state["kind"]
    if kind == "norm_rope":
        return _norm_rope(s, s["q"], s["wq"]), _norm_rope(s, s["k"], s["wk"])
    if kind == "norm_rope_grad":
        (dq, dwq), (dk, dwk) = _norm_rope_grad(s, s["gq"], s["q"], s["wq"]), _norm_rope_grad(s, s["gk"], s["k"], s["wk"])
        return dq, dk, dwq, dwk
    return {"append": _append_plain, "attend": _attend_plain, "verify": _verify_plain}[kind](s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind == "verify":
        n, k, v = case["seqs"], case["drafts"], case["vocab"]
        rows = 2 if case["draft_probs"] else 1  # one row of the target and, behind a rejection, one of the draft
        return {"bytes": n * (rows * v * 4 + k * 16 + (k + 1) * 4 + 12), "flops": 3.0 * n * v}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if kind in ("norm_rope", "norm_rope_grad"):
        rows = case["real"] * (hq + hkv) * d
        every = case["n"] * (hq + hkv) * d
        table = min(case["real"], 8192) * case["rot"] * 4 + 4 * case["n"]
        if kind == "norm_rope":
            return {"bytes": 2 * rows + 2 * every + table, "flops": 8.0 * rows}
        g = 2 if case["grad_type"] == "bf16" else 4
        return {"bytes": (g + (2 if case["norm"] else 0)) * rows + g * every + table, "flops": 16.0 * rows}
    q_lens, kv_lens = _lens(case)
    n = sum(q_lens)
    table = 4 * sum(len(r) for r in _pages(case)[0]) + 8 * case["seqs"]
    if kind == "append":
        return {"bytes": 4 * n * (hq + 2 * hkv) * d + 4 * min(n, max(kv_lens)) * d + table,
                "flops": 8.0 * n * (hq + hkv) * d}
    w, p = case["window"], case["page"]
    pairs, used = 0, {}
    for s, (a, b) in enumerate(zip(q_lens, kv_lens)):
        first = max(0, b - a - w + 1) if w else 0
        pairs += sum(min(b - a + i + 1, w) if w else b - a + i + 1 for i in range(a))
        for x, page in enumerate(_pages_of(case)[s]):
            used[page] = max(used.get(page, 0), min(p, b - x * p) if (x + 1) * p > first else 0)
    return {"bytes": 4 * sum(used.values()) * hkv * d + 4 * n * hq * d + 4 * n * hq + table,
            "flops": 4.0 * pairs * hq * d}


def _pages_of(case, kept={}):
    key = tuple(sorted((k, v) for k, v in case.items() if k != "name"))
    if kept.get("key") != key:
        kept.update(key=key, rows=_pages(case)[0])
    return kept["rows"]


# ------------------------------------------------------------------ the same in 64 bits

def _turn(x, pos, rot, interleaved):
    """x [n, h, d] in 64 bits with the pairs of its first `rot` values as complex numbers turned by pos x frequency."""
    angles = _table(8192 if pos.numel() == 0 else max(1, int(pos.max()) + 1), rot)[pos].double()
    z = torch.complex(angles[:, :rot // 2], angles[:, rot // 2:])[:, None]
    head, rest = x[..., :rot], x[..., rot:]
    pairs = head.unflatten(-1, (rot // 2, 2)) if interleaved else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    t = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    return torch.cat([(t if interleaved else t.transpose(-1, -2)).flatten(-2), rest], -1)


def _exact_rope(x, w, pos, rot, interleaved):
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
    return _turn(x, pos, rot, interleaved)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "verify":
        return _exact_verify(s)
    double = lambda t: None if t is None else t.double()  # noqa: E731
    if kind in ("norm_rope", "norm_rope_grad"):
        n = case["real"]
        pos = s["positions"][:n].long()
        got, weights = [], []
        for x, w, g in (("q", "wq", "gq"), ("k", "wk", "gk")):
            v = s[x][:n].double().requires_grad_()
            t = None if s[w] is None else s[w].double().requires_grad_()
            y = _exact_rope(v, t, pos, case["rot"], case["interleaved"])
            out = torch.zeros(s[x].shape, dtype=torch.float64, device="cuda")
            if kind == "norm_rope":
                out[:n] = y.detach()
            elif t is None:
                out[:n] = torch.autograd.grad(y, v, s[g][:n].double())[0]
                weights.append(None)
            else:
                out[:n], dw = torch.autograd.grad(y, (v, t), s[g][:n].double())
                weights.append(dw)
            got.append(out)
        return tuple(got) if kind == "norm_rope" else (*got, *weights)
    q_lens, kv_lens = _lens(case)
    p, start = case["page"], np.cumsum([0] + q_lens)
    pages = s["pages"].long()
    if kind == "append":
        pos = torch.cat([torch.arange(b - a, b) for a, b in zip(q_lens, kv_lens)]).cuda()
        q = _exact_rope(s["q"].double(), double(s["wq"]), pos, case["d"], False)
        k = _exact_rope(s["k"].double(), double(s["wk"]), pos, case["d"], False)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for i, (a, b) in enumerate(zip(q_lens, kv_lens)):
            at = torch.arange(b - a, b, device="cuda")
            kc[pages[i, at // p], :, at % p] = k[start[i]:start[i + 1]]
            vc[pages[i, at // p], :, at % p] = s["v"][start[i]:start[i + 1]].double()
        return q, kc, vc
    hq, d, g = case["hq"], case["d"], case["hq"] // case["hkv"]
    if 4.0 * sum(a * b for a, b in zip(q_lens, kv_lens)) * hq * d > 4e12:
        return None
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(zip(q_lens, kv_lens)):
        rows = slice(int(start[i]), int(start[i + 1]))
        j = torch.arange(b, device="cuda")
        pos = torch.arange(b - a, b, device="cuda")[:, None]
        hidden = (j > pos) | (j <= pos - case["window"] if case["window"] else j > pos)
        for h in range(hq):
            k, v = (c[pages[i, j // p], h // g, j % p].double() for c in (s["k_cache"], s["v_cache"]))
            x = torch.where(hidden, -math.inf, s["q"][rows, h].double() @ k.T / math.sqrt(d))
            o[rows, h], lse[rows, h] = torch.softmax(x, -1) @ v, torch.logsumexp(x, -1)
    return o, lse


def _exact_verify(s):
    p, u, u_next, x = (s[k].cpu().numpy() for k in ("target", "u_accept", "u_next", "tokens"))
    q = None if s["draft"] is None else s["draft"].cpu().numpy()
    n, k = x.shape
    out, counts = np.full((n, k + 1), -1, dtype=np.int32), np.zeros(n, dtype=np.int32)
    for r, most in enumerate(s["n_drafts"].tolist()):
        i = 0
        while i < most:
            beside = 1.0 if q is None else float(q[r, i, x[r, i]])
            if not float(u[r, i]) * beside < float(p[r, i, x[r, i]]):
                break
            out[r, i] = x[r, i]
            i += 1
        weights = p[r, i].astype(np.float64)
        if i < most:
            left = weights.copy()
            if q is None:
                left[x[r, i]] = 0
            else:
                left = np.maximum(left - q[r, i].astype(np.float64), 0)
            weights = left if left.sum() > 0 else weights
        sums = np.cumsum(weights)
        out[r, i] = min(int(np.searchsorted(sums, float(u_next[r]) * sums[-1], side="right")), int(np.nonzero(weights)[0][-1]))
        counts[r] = i
    return torch.from_numpy(out), torch.from_numpy(counts)
