"""Operators of a sampling step that drafts trees of tokens, as cases to measure.

A policy that is trained on packed trees is sampled from a paged cache.  A step
that drafts a tree of continuations for each sequence, and a batch whose
prompts are sampled several times, need beside the attention over the cache:

- ``attend``: attention of each sequence's drafted tree over its pages, where a
  token sees what is cached before the tree, its ancestors in it and itself;
- ``sample``: the next token of each row of logits, with temperature, top-k,
  top-p and min-p, from given uniform numbers, and its log-probability;
- ``round``: what surrounds the model in a step: the tree's positions and masks
  from its parents; the path that the sampled tokens follow through it; and the
  cache with that path's keys and values moved to where the sequence goes on;
- ``pages``: between batches: pages of sequences that ended go back, new
  sequences get theirs, and samples of a prompt start as its forks, with whole
  pages shared and the last, partly filled one copied.

``run`` computes them by elementary torch operations, or through the package
where ``own`` is true.  ``exact`` gives the same outputs in 64 bits, written
apart from both.
"""
import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ the cases

def _sample(name, rows, vocab, type_, temperature, top_k, top_p, min_p, mixed):
    return {"name": name, "kind": "sample", "rows": rows, "vocab": vocab, "type": type_, "temperature": temperature,
            "top_k": top_k, "top_p": top_p, "min_p": min_p, "mixed": mixed}


def _attend(name, seqs, q_low, q_high, kv_low, kv_high, hq, hkv, d, page, window):
    return {"name": name, "kind": "attend", "seqs": seqs, "q_low": q_low, "q_high": q_high, "kv_low": kv_low,
            "kv_high": kv_high, "hq": hq, "hkv": hkv, "d": d, "page": page, "window": window}


def _round(name, seqs, q_low, q_high, kv_low, kv_high, hkv, d, page, layers):
    return {"name": name, "kind": "round", "seqs": seqs, "q_low": q_low, "q_high": q_high, "kv_low": kv_low,
            "kv_high": kv_high, "hkv": hkv, "d": d, "page": page, "layers": layers}


def _pages(name, kept, prompts, samples, kv_low, kv_high, hkv, d, page, layers, spare):
    return {"name": name, "kind": "pages", "kept": kept, "prompts": prompts, "samples": samples, "kv_low": kv_low,
            "kv_high": kv_high, "hkv": hkv, "d": d, "page": page, "layers": layers, "spare": spare}


def listed():
    return [
        # one request, the tokenised workloads' ids: the call's latency
        _sample("sample one request", 1, 32000, "f32", 0.7, 40, 0.95, 0.0, False),
        # a decode step of 8 prompts x 8 samples as policy training wants it: the policy's own distribution
        _sample("sample GRPO step", 64, 151936, "bf16", 1.0, 0, 1.0, 0.0, False),
        # a server's batch: every request with its own temperature, top-k, top-p and min-p
        _sample("sample mixed requests", 64, 151936, "f32", 0.8, 50, 0.9, 0.05, True),
        # a token for every row of 16 sequences' drafted trees
        _sample("sample tree rows", 499, 32000, "bf16", 0.9, 0, 0.9, 0.0, False),
        # 64 samples with 8 drafted tokens each
        _attend("attend GRPO drafts", 64, 8, 8, 300, 3000, 32, 8, 128, 16, 0),
        # larger trees of 16 sequences, 20 to 64 tokens
        _attend("attend ragged trees", 16, 20, 64, 1000, 8000, 32, 8, 128, 32, 0),
        # one long agentic trajectory: the work has to be split along the keys
        _attend("attend long", 1, 48, 48, 130001, 130001, 16, 2, 128, 64, 0),
        # one sequence's tree in the tiny workload's heads: latency
        _round("round one sequence", 1, 16, 16, 700, 700, 4, 64, 16, 2),
        # the ragged trees again, over a cache of eight layers
        _round("round ragged trees", 64, 20, 64, 300, 3000, 8, 128, 16, 8),
        # two prompts come in beside eight sequences
        _pages("pages small", 8, 2, 4, 300, 1000, 4, 64, 16, 1, 500),
        # 8 prompts x 8 samples over eight layers' caches
        _pages("pages GRPO", 16, 8, 8, 256, 1024, 8, 128, 64, 8, 100),
        # a server's pool: many sequences, small pages, one layer's cache
        _pages("pages pool", 500, 64, 8, 100, 4000, 1, 64, 16, 1, 40000),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["sample", "sample", "attend", "attend", "round", "pages"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if kind == "sample":
        vocab = _log(rng, 1000, 151936)
        c = _sample("", _log(rng, 1, min(600, max(1, 9700000 // vocab))), vocab, rng.choice(["bf16", "f32"]),
                    round(rng.uniform(0.3, 1.3), 3), rng.choice([0, 0, 1, 20, 50, 1000]),
                    rng.choice([1.0, 1.0, 0.5, 0.9, 0.97]), rng.choice([0.0, 0.0, 0.05, 0.2]), rng.random() < 0.3)
    elif kind == "attend":
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
        seqs = _log(rng, 1, 64)
        high = _log(rng, 1, max(1, min(200, 1000 // seqs)))
        kv = high + _log(rng, 1, max(2, min(120000 // seqs, 90000000 // (seqs * high * hq))))
        c = _attend("", seqs, rng.randint(1, high), high, rng.randint(high, kv), kv, hq, hkv, d, page,
                    rng.choice([0, 0, 0, 100, 1000]))
    elif kind == "round":
        seqs = _log(rng, 1, 64)
        high = _log(rng, 1, 200)
        kv = high + _log(rng, 1, max(2, 130000 // seqs))
        c = _round("", seqs, rng.randint(1, high), high, rng.randint(high, kv), kv, hkv, d, page, rng.randint(1, 4))
    else:
        prompts = _log(rng, 1, 32)
        high = _log(rng, 2, 3000)
        c = _pages("", _log(rng, 1, 200), prompts, rng.randint(1, 8), rng.randint(1, high), high, rng.choice([1, 2]), 64,
                   page, rng.randint(1, 2), _log(rng, 400, 20000))
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs

def _lens(case):
    """New tokens and cached tokens (the new ones among them) of each sequence: the case's own, whatever the seed."""
    r = random.Random(1)
    q = [r.randint(case["q_low"], case["q_high"]) for _ in range(case["seqs"])]
    return q, [max(a, r.randint(case["kv_low"], case["kv_high"])) for a in q]


def _parents(n, r):
    """A drafted tree in the order in which it is drafted: row 0 the last sampled token, then its continuations, two to
    four of each."""
    return [-1] + [r.randint((i - 1) // 4, (i - 1) // 2) for i in range(1, n)]


def _rows_of_pages(lens, page):
    """Numbers for the pages of each sequence, and how many there are."""
    rows, count = [], 0
    for n in lens:
        need = -(-n // page)
        rows.append(list(range(count, count + need)))
        count += need
    return rows, count


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_sample(s, g, r):
    n, v = s["rows"], s["vocab"]
    # what a policy's head gives: a broad floor of the vocabulary, and a few dozen tokens above it
    x = 2.5 * _normal(g, n, v)
    at = torch.randint(0, v, (n, 24), generator=g, device="cuda")
    x.scatter_add_(1, at, 4 + 10 * _uniform(g, n, 24))
    s["logits"] = x.to(torch.bfloat16) if s["type"] == "bf16" else x
    s["u"] = _uniform(g, n)
    if s["mixed"]:
        # requests of their own kinds, greedy ones among them
        pick = lambda of: [r.choice(of) for _ in range(n)]  # noqa: E731
        t = s["temperature"]
        s["temperature"] = torch.tensor([r.choice([0.0, t, t, r.uniform(0.5, 1.2)]) for _ in range(n)], device="cuda")
        s["top_k"] = _i32(pick([0, s["top_k"], 20]))
        s["top_p"] = torch.tensor(pick([1.0, s["top_p"], 0.95]), device="cuda")
        s["min_p"] = torch.tensor(pick([0.0, s["min_p"]]), device="cuda")


def _prepare_tree(s, g, r):
    """The batch of `attend` and `round`: pages, offsets, lengths, parents; caches of `layers`."""
    q_lens, kv_lens = _lens(s)
    page, n = s["page"], sum(q_lens)
    rows, count = _rows_of_pages(kv_lens, page)
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    width = max(len(x) for x in rows)
    s["pages"] = order[torch.tensor([x + [0] * (width - len(x)) for x in rows], device="cuda")].contiguous()
    s["offsets"] = _i32([0] + list(np.cumsum(q_lens)))
    s["kv_lens"] = _i32(kv_lens)
    s["max_q"], s["max_kv"], s["n"] = max(q_lens), max(kv_lens), n
    trees = [_parents(a, r) for a in q_lens]
    s["parents"] = _i32([p for t in trees for p in t])
    shape = (count, s["hkv"], page, s["d"])
    if s["kind"] == "attend":
        s["k_cache"], s["v_cache"] = (_normal(g, *shape).to(torch.bfloat16) for _ in range(2))
        s["q"] = _normal(g, n, s["hq"], s["d"]).to(torch.bfloat16)
        # made once a step, for all layers
        depth, seen = [], []
        words = -(-s["max_q"] // 32)
        for t, b in zip(trees, kv_lens):
            deep, masks = [], []
            for i, p in enumerate(t):
                deep.append(0 if p < 0 else deep[p] + 1)
                masks.append((1 << i) | (0 if p < 0 else masks[p]))
            if s["window"]:
                masks = [sum(1 << j for j in range(i + 1) if m >> j & 1 and deep[i] - deep[j] < s["window"])
                         for i, m in enumerate(masks)]
            depth += [b - len(t) + x for x in deep]
            seen += [[m >> 32 * w & 0xffffffff for w in range(words)] for m in masks]
        s["positions"] = _i32(depth)
        s["masks"] = torch.tensor(seen, dtype=torch.int64, device="cuda").to(torch.int32)
        return
    s["k_cache"], s["v_cache"] = (torch.randn((s["layers"], *shape), generator=g, device="cuda", dtype=torch.bfloat16)
                                  for _ in range(2))
    # the drafter proposes different tokens behind the same one; the policy's own choice is among them, most times
    tokens, sampled = [], []
    for t in trees:
        x = [1000 * i + r.randint(0, 999) for i in range(len(t))]
        y = [r.randint(10 ** 6, 2 * 10 ** 6) for _ in t]
        path, at = [0], 0
        while r.random() < 0.8:
            below = [i for i, p in enumerate(t) if p == at]
            if not below:
                break
            at = r.choice(below)
            path.append(at)
        # a pass can be made again on the caches that it left: no place is written that the path is read from
        while any(p != i and p < len(path) for i, p in enumerate(path)):
            path.pop()
        for a, b in zip(path, path[1:]):
            y[a] = x[b]
        tokens += x
        sampled += y
    s["tokens"], s["sampled"] = _i32(tokens), _i32(sampled)


def _prepare_pages(s, g, r):
    kept, prompts, samples, page = s["kept"], s["prompts"], s["samples"], s["page"]
    rows = kept + prompts * (1 + samples)
    lengths = random.Random(1)  # the case's own, whatever the seed
    lens, new = ([lengths.randint(s["kv_low"], s["kv_high"]) for _ in range(n)] for n in (kept, prompts))
    need = [-(-n // page) for n in lens + new]
    width = max(need) + 1
    count = sum(need) + prompts * samples + s["spare"]
    order = list(range(count))
    r.shuffle(order)
    table = np.full((rows, width), -1, np.int32)
    for i in range(kept):
        table[i, :need[i]] = order[:need[i]]
        del order[:need[i]]
    refs = np.zeros(count, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    rest = [0] * (prompts * samples)
    s["pages"], s["refs"] = _i32(table), _i32(refs)
    s["retired"], s["admitted"] = _i32(lens + [0] * prompts + rest), _i32(lens + new + rest)
    s["kv_lens"] = s["retired"].clone()
    s["src"] = _i32([kept + i for i in range(prompts) for _ in range(samples)])
    s["dst"] = _i32([kept + prompts + i for i in range(prompts * samples)])
    shape = (s["layers"], count, s["hkv"], page, s["d"])
    s["k_cache"], s["v_cache"] = (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    r = random.Random(int(seed))
    s = dict(case)
    {"sample": _prepare_sample, "attend": _prepare_tree, "round": _prepare_tree, "pages": _prepare_pages}[s["kind"]](s, g, r)
    return s


# ------------------------------------------------------------------ the operators

def _column(x, rows, dtype):
    return (x if isinstance(x, torch.Tensor) else torch.full((rows,), x, device="cuda")).to(dtype)[:, None]


def _sample_plain(s):
    # in 64 bits: a draw lies next to a border of running sums
    n, v = s["logits"].shape
    t, p, least = (_column(s[k], n, torch.float32).double() for k in ("temperature", "top_p", "min_p"))
    k = _column(s["top_k"], n, torch.int64)
    k = torch.where(t == 0, 1, torch.where(k <= 0, v, k))
    t = torch.where(t == 0, 1.0, t)
    x = s["logits"].double()
    rank = torch.arange(v, device="cuda")
    if s["mixed"] or s["top_k"] or s["top_p"] < 1:
        x, at = torch.sort(x, dim=1, descending=True, stable=True)
        w = ((x - x[:, :1]) / t).exp()
        w = torch.where(rank < k, w, 0.0)
        before = w.cumsum(1) - w
        w = torch.where((rank == 0) | (p >= 1) | (before < p * w.sum(1, keepdim=True)), w, 0.0)
        w = torch.empty_like(w).scatter_(1, at, w)
    else:
        w = ((x - x.amax(1, keepdim=True)) / t).exp()
    w = torch.where(w >= least, w, 0.0)
    sums = w.cumsum(1)
    past = (sums > s["u"].double()[:, None] * sums[:, -1:]) & (w > 0)
    token = torch.where(past, rank, v).amin(1)
    last = torch.where(w > 0, rank, -1).amax(1)
    token = torch.where(token < v, token, last)
    logp = (w.gather(1, token[:, None])[:, 0] / sums[:, -1]).log()
    return token.to(torch.int32), logp.float()


def _token_places(s, n):
    """For each new token: its sequence, its number among the sequence's new tokens, and the sequence's tokens before."""
    i = torch.arange(n, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"][1:], i, right=True)
    base = s["kv_lens"] - (s["offsets"][1:] - s["offsets"][:-1])
    return seq, (i - s["offsets"][seq]).long(), base[seq]


def _bits(masks, count):
    j = torch.arange(count, device="cuda")
    return (masks[:, j // 32] >> (j % 32)) & 1 != 0


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
    base = (s["kv_lens"] - (s["offsets"][1:] - s["offsets"][:-1]))[:, None]
    j = torch.arange(lk, device="cuda")
    seen = (j < base)[:, None].expand(nseq, lq, lk)
    if s["window"]:
        seen = seen & (j > s["positions"][at][..., None] - s["window"])
    drafted = (j - base)[:, None].expand(nseq, lq, lk)               # number of the key's token among the new ones
    bit = _bits(s["masks"], lq)[at].gather(2, drafted.clamp(0, lq - 1).long())
    seen = seen | ((drafted >= 0) & (drafted <= torch.arange(lq, device="cuda")[:, None]) & bit)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(nseq, hkv, g * lq, lk) @ keys(s["v_cache"])).view(nseq, hkv, g, lq, d) / total.clamp(min=1e-30)
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(nseq, lq, hq, d)[seq, local]
    lse = lse.permute(0, 3, 1, 2).reshape(nseq, lq, hq)[seq, local]
    return o.to(torch.bfloat16), lse


def _round_plain(s):
    n, nseq, lq, page = s["n"], s["seqs"], s["max_q"], s["page"]
    seq, local, base = _token_places(s, n)

    def padded(x, fill):
        return torch.full((nseq, lq), fill, dtype=torch.long, device="cuda").index_put_((seq, local), x.long())

    # ancestors: the closure of the parents, by squaring
    parent = padded(s["parents"], -1)
    i = torch.arange(lq, device="cuda")
    edge = (parent[:, :, None] == i).float()
    above = edge + torch.eye(lq, device="cuda")
    for _ in range(max(1, (lq - 1).bit_length())):
        above = ((above @ above) > 0).float()
    positions = base + (above.sum(2) - 1)[seq, local].to(torch.int32)
    words = -(-lq // 32)
    bits = torch.nn.functional.pad(above, (0, 32 * words - lq)).view(nseq, lq, words, 32).to(torch.int64)
    masks = (bits << torch.arange(32, device="cuda")).sum(3)[seq, local].to(torch.int32)

    # a token is on the path when it and every ancestor are the first of their parent's children with the sampled token
    tokens, sampled = padded(s["tokens"], -1), padded(s["sampled"], -2)
    fits = (parent[:, None] == i[:, None]) & (tokens[:, None] == sampled[:, :, None])   # [seq, parent, child]
    first = torch.where(fits, i, lq).amin(2)
    stands = (first.gather(1, parent.clamp(min=0)) == i) & (parent >= 0)
    stands[:, 0] = True
    on = ((above @ (~stands).float()[..., None])[..., 0] == 0) & (i < (s["offsets"][1:] - s["offsets"][:-1])[:, None])
    count = on.sum(1)
    path = torch.where(on, i, lq).sort(1).values
    there = i < count[:, None]
    path = torch.where(there, path, -1)
    emitted = torch.where(there, sampled.gather(1, path.clamp(min=0)), -1)

    # the path's keys and values, read before they are written
    start = (s["kv_lens"] - (s["offsets"][1:] - s["offsets"][:-1])).long()[:, None]
    which, to = there.nonzero(as_tuple=True)
    old, new = (start + path)[which, to], (start + i)[which, to]
    for cache in (s["k_cache"], s["v_cache"]):
        x = cache[:, s["pages"][which, old // page].long(), :, old % page]
        cache[:, s["pages"][which, new // page].long(), :, new % page] = x
    lens = start[:, 0] + count
    t32 = lambda x: x.to(torch.int32)  # noqa: E731
    return positions, masks, t32(emitted), t32(path), t32(count), t32(lens), s["k_cache"], s["v_cache"]


def _resize_plain(s):
    pages, refs, page = s["pages"], s["refs"], s["page"]
    j = torch.arange(pages.shape[1], device="cuda")
    need = ((s["kv_lens"] + page - 1) // page)[:, None]
    drop = (pages >= 0) & (j >= need)
    refs.index_add_(0, pages[drop].long(), torch.full((1,), -1, dtype=torch.int32, device="cuda").expand(int(drop.sum())))
    pages[drop] = -1
    want = (pages < 0) & (j < need)
    free = (refs == 0).nonzero()[:, 0]
    got = free[:int(want.sum())]
    pages[want] = got.to(torch.int32)
    refs[got] = 1
    return torch.full((1,), len(free) - len(got), dtype=torch.int32, device="cuda")


def _fork_plain(s):
    pages, refs, page, lens = s["pages"], s["refs"], s["page"], s["kv_lens"]
    src, dst = s["src"].long(), s["dst"].long()
    old = pages[dst]
    refs.index_add_(0, old[old >= 0].long(), torch.full((1,), -1, dtype=torch.int32, device="cuda").expand(int((old >= 0).sum())))
    whole, part = lens[src] // page, lens[src] % page
    j = torch.arange(pages.shape[1], device="cuda")
    row = torch.where(j < whole[:, None], pages[src], -1)
    refs.index_add_(0, row[row >= 0].long(), torch.ones(1, dtype=torch.int32, device="cuda").expand(int((row >= 0).sum())))
    some = (part > 0).nonzero()[:, 0]
    free = (refs == 0).nonzero()[:, 0]
    got = free[:len(some)]
    last = pages[src[some], whole[some].long()].long()
    row[some, whole[some].long()] = got.to(torch.int32)
    refs[got] = 1
    pages[dst] = row
    lens[dst] = lens[src]
    keep = (torch.arange(page, device="cuda") < part[some, None])[:, None, :, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, got] = torch.where(keep, cache[:, last], cache[:, got])
    return torch.full((1,), len(free) - len(got), dtype=torch.int32, device="cuda")


def _pages_plain(s):
    s["kv_lens"].copy_(s["retired"])
    _resize_plain(s)
    s["kv_lens"].copy_(s["admitted"])
    room = _resize_plain(s)
    left = _fork_plain(s)
    return s["pages"], s["refs"], s["kv_lens"], room, left, s["k_cache"], s["v_cache"]


def _run_own(s):
    import prefix_shared_tree_attention_gb300 as tpa
    kind = s["kind"]
    if kind == "sample":
        return tpa.sample_tokens(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                 min_p=s["min_p"])
    if kind == "attend":
        return tpa.paged_attn_tree_fwd(s["k_cache"], s["v_cache"], s["pages"], s["offsets"], s["kv_lens"], s["q"],
                                       s["masks"], max_q_len=s["max_q"], window=s["window"], positions=s["positions"])
    if kind == "round":
        positions, masks = tpa.draft_masks(s["parents"], s["offsets"], s["kv_lens"], max_q_len=s["max_q"])
        tokens, path, count = tpa.accept_drafts(s["parents"], s["offsets"], s["tokens"], s["sampled"], max_path=s["max_q"])
        lens = tpa.paged_compact(s["k_cache"], s["v_cache"], s["pages"], s["offsets"], s["kv_lens"], path, count)
        return positions, masks, tokens, path, count, lens, s["k_cache"], s["v_cache"]
    s["kv_lens"].copy_(s["retired"])
    tpa.paged_resize(s["pages"], s["kv_lens"], s["refs"], s["page"])
    s["kv_lens"].copy_(s["admitted"])
    room = tpa.paged_resize(s["pages"], s["kv_lens"], s["refs"], s["page"])
    left = tpa.paged_fork(s["k_cache"], s["v_cache"], s["pages"], s["kv_lens"], s["refs"], s["src"], s["dst"])
    return s["pages"], s["refs"], s["kv_lens"], room, left, s["k_cache"], s["v_cache"]


def run(state):
    if own:
        return _run_own(state)
    return {"sample": _sample_plain, "attend": _attend_plain, "round": _round_plain, "pages": _pages_plain}[state["kind"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind == "sample":
        n, v = case["rows"], case["vocab"]
        return {"bytes": n * (v * (2 if case["type"] == "bf16" else 4) + 4 + 8 + (16 if case["mixed"] else 0)), "flops": 3.0 * n * v}
    if kind == "pages":
        # the lengths' distribution, not a seed's: a page table entry read and written for each page that moves, the
        # counts once, half a page a prompt read and a sample written
        mean, page = (case["kv_low"] + case["kv_high"]) / 2, case["page"]
        forks, each = case["prompts"] * case["samples"], mean / page
        moved = (case["prompts"] + forks) * each
        pool = (case["kept"] + case["prompts"]) * each + forks + case["spare"]
        half = case["layers"] * 2 * case["hkv"] * (page / 2) * case["d"] * 2
        return {"bytes": int(3 * 8 * moved + 4 * pool + (case["prompts"] + forks) * half), "flops": float(int(moved) + 1)}
    q_lens, kv_lens = _lens(case)
    n, p, hkv, d = sum(q_lens), case["page"], case["hkv"], case["d"]
    words = -(-max(q_lens) // 32)
    if kind == "round":
        # a path of three tokens, two of which move: read and written, keys and values of all layers
        moves = 2 * case["seqs"]
        return {"bytes": n * (4 + 4 + 4 + 4 + 4 * words) + 24 * case["seqs"] + moves * 2 * 2 * case["layers"] * hkv * d * 2,
                "flops": float(n * words)}
    hq, w = case["hq"], case["window"]
    table = 4 * sum(-(-b // p) for b in kv_lens) + 8 * case["seqs"]
    keys = [a + min(b - a, w) if w else b for a, b in zip(q_lens, kv_lens)]
    pairs = sum(a * (b - a) + 5 * a for a, b in zip(q_lens, keys))   # a drafted token has a handful of ancestors
    return {"bytes": 4 * sum(keys) * hkv * d + 4 * n * hq * d + 4 * n * hq + 4 * n * words + table,
            "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------------ the same in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "attend": _exact_attend, "round": _exact_round, "pages": _exact_pages}[case["kind"]](s)


def _exact_sample(s):
    x, u = s["logits"].double().cpu().numpy(), s["u"].double().cpu().numpy()
    n, v = x.shape
    row = lambda a: a.cpu().numpy() if isinstance(a, torch.Tensor) else np.full(n, a)  # noqa: E731
    t, k = row(s["temperature"]).astype(np.float32), row(s["top_k"])
    p, least = row(s["top_p"]).astype(np.float32), row(s["min_p"]).astype(np.float32)
    tokens, logp = np.zeros(n, np.int32), np.zeros(n)
    for i in range(n):
        if t[i] == 0:
            tokens[i] = int(x[i].argmax())
            continue
        w = np.exp((x[i] - x[i].max()) / float(t[i]))
        if 0 < k[i] < v or p[i] < 1:
            order = np.argsort(-x[i], kind="stable")
            order = order[:k[i]] if 0 < k[i] < v else order
            if p[i] < 1:
                sums = np.cumsum(w[order])
                order = order[:int(np.searchsorted(sums, float(p[i]) * sums[-1])) + 1]
            kept = np.zeros(v, bool)
            kept[order] = True
            w = np.where(kept, w, 0.0)
        w = np.where(w >= float(least[i]), w, 0.0)
        sums = np.cumsum(w)
        at = min(int(np.searchsorted(sums, u[i] * sums[-1], side="right")), int(np.nonzero(w)[0][-1]))
        tokens[i], logp[i] = at, math.log(w[at] / sums[-1])
    return torch.from_numpy(tokens), torch.from_numpy(logp)


def _exact_attend(s):
    q_lens, kv_lens = _lens(s)
    page, hq, d, g, w = s["page"], s["hq"], s["d"], s["hq"] // s["hkv"], s["window"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    pages, parents, first = s["pages"].long(), s["parents"].tolist(), 0
    for i, (a, b) in enumerate(zip(q_lens, kv_lens)):
        # which keys a token sees, by walking up from it
        seen = np.zeros((a, b), bool)
        for t in range(a):
            up, steps = t, 0
            while up >= 0:
                if not w or steps < w:
                    seen[t, b - a + up] = True
                up, steps = parents[first + up], steps + 1
            steps -= 1                                                # the token's depth
            seen[t, max(0, b - a + steps - w + 1) if w else 0:b - a] = True
        hidden = ~torch.from_numpy(seen).cuda()
        rows = slice(first, first + a)
        j = torch.arange(b, device="cuda")
        for h in range(hq):
            k, v = (c[pages[i, j // page], h // g, j % page].double() for c in (s["k_cache"], s["v_cache"]))
            x = torch.where(hidden, -math.inf, s["q"][rows, h].double() @ k.T / math.sqrt(d))
            o[rows, h], lse[rows, h] = torch.softmax(x, -1) @ v, torch.logsumexp(x, -1)
        first += a
    return o, lse


def _exact_round(s):
    q_lens, kv_lens = _lens(s)
    page, words, most = s["page"], -(-s["max_q"] // 32), s["max_q"]
    parents, tokens, sampled = (s[k].tolist() for k in ("parents", "tokens", "sampled"))
    pages = s["pages"].cpu()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    positions, masks, first = [], [], 0
    emitted, paths = (np.full((s["seqs"], most), -1, np.int32) for _ in range(2))
    counts, lens = (np.zeros(s["seqs"], np.int32) for _ in range(2))
    for i, (a, b) in enumerate(zip(q_lens, kv_lens)):
        up = parents[first:first + a]
        for t in range(a):
            chain = [t]
            while up[chain[-1]] >= 0:
                chain.append(up[chain[-1]])
            positions.append(b - a + len(chain) - 1)
            mask = sum(1 << j for j in chain)
            masks.append([mask >> 32 * w & 0xffffffff for w in range(words)])
        path = [0]
        while True:
            y = sampled[first + path[-1]]
            emitted[i, len(path) - 1] = y
            below = [t for t in range(a) if up[t] == path[-1] and tokens[first + t] == y]
            if not below:
                break
            path.append(below[0])
        paths[i, :len(path)], counts[i], lens[i] = path, len(path), b - a + len(path)
        rows = [(k[:, pages[i, (b - a + t) // page], :, (b - a + t) % page].clone(),
                 v[:, pages[i, (b - a + t) // page], :, (b - a + t) % page].clone()) for t in path for k, v in [(kc, vc)]]
        for t, (k, v) in enumerate(rows):
            at = b - a + t
            kc[:, pages[i, at // page], :, at % page] = k
            vc[:, pages[i, at // page], :, at % page] = v
        first += a
    whole = lambda x: torch.from_numpy(np.asarray(x))  # noqa: E731
    return (whole(np.array(positions, np.int32)), whole(np.array(masks, np.int64).astype(np.uint32).view(np.int32)),
            whole(emitted), whole(paths), whole(counts), whole(lens), kc, vc)


def _exact_pages(s):
    page = s["page"]
    table, refs = s["pages"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()
    rows = [[x for x in t if x >= 0] for t in table.tolist()]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()

    def resize(lens):
        need = [-(-n // page) for n in lens]
        for t, n in zip(rows, need):
            while len(t) > n:
                refs[t.pop()] -= 1
        free = iter(np.nonzero(refs == 0)[0].tolist())
        for t, n in zip(rows, need):
            while len(t) < n:
                t.append(next(free))
                refs[t[-1]] = 1
        return int((refs == 0).sum())

    lens = s["retired"].tolist()
    resize(lens)
    lens = s["admitted"].tolist()
    room = resize(lens)
    src, dst = s["src"].tolist(), s["dst"].tolist()
    for b in dst:
        while rows[b]:
            refs[rows[b].pop()] -= 1
    for a, b in zip(src, dst):
        rows[b] = rows[a][:lens[a] // page]
        refs[rows[b]] += 1
        lens[b] = lens[a]
    free = iter(np.nonzero(refs == 0)[0].tolist())
    for a, b in zip(src, dst):
        part = lens[a] % page
        if part:
            new, old = next(free), rows[a][lens[a] // page]
            rows[b] = rows[b] + [new]
            refs[new] = 1
            for c in (kc, vc):
                c[:, new, :, :part] = c[:, old, :, :part]
    table[:] = -1
    for t, x in zip(table, rows):
        t[:len(x)] = x
    one = lambda x: torch.tensor([x], dtype=torch.int32)  # noqa: E731
    return (torch.from_numpy(table), torch.from_numpy(refs), torch.tensor(lens, dtype=torch.int32), one(room),
            one(int((refs == 0).sum())), kc, vc)
