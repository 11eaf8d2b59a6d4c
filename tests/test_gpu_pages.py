"""The pages of a cache (tpa_paged_resize, tpa_paged_fork): tables, counts, lengths and copied values equal to the oracle's."""
import numpy as np
import pytest
import torch

from oracle.pages import Pool
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


class Both:
    """The device's state beside the oracle's, guarded."""

    def __init__(self, n_pages, n_rows, width, page, layers=0, hkv=2, d=64, pad=0):
        self.pool = Pool(n_pages, n_rows, page)
        self.bt, table = guarded((n_rows, width + pad), torch.int32)
        table.fill_(-1)
        self.table = table
        self.pages = table[:, :width]
        self.br, self.refs = guarded((n_pages,), torch.int32)
        self.bl, self.lens = guarded((n_rows,), torch.int32)
        self.bf, self.left = guarded((1,), torch.int32)
        self.refs.zero_()
        self.lens.zero_()
        self.page = page
        if layers:
            g = torch.Generator().manual_seed(1)
            self.k, self.v = (torch.randn((layers, n_pages, hkv, page, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))

    def check(self, left):
        for b, what in ((self.bt, "pages"), (self.br, "refs"), (self.bl, "lens"), (self.bf, "n_free")):
            check_guards(b, what)
        width = self.pages.shape[1]
        assert self.left.item() == left
        assert self.refs.tolist() == self.pool.refs
        assert self.lens.tolist() == self.pool.lens
        assert self.pages.tolist() == [r + [-1] * (width - len(r)) for r in self.pool.rows]
        assert (self.table[:, width:] == -1).all()

    def resize(self, tpa, lens):
        self.lens.copy_(_i32(lens))
        tpa.paged_resize(self.pages, self.lens, self.refs, self.page, out=self.left)
        self.check(self.pool.resize(lens))

    def fork(self, tpa, src, dst):
        before = self.k.clone(), self.v.clone()
        tpa.paged_fork(self.k, self.v, self.pages, self.lens, self.refs, _i32(src).cuda(), _i32(dst).cuda(), out=self.left)
        left, copies = self.pool.fork(src, dst)
        self.check(left)
        for c, b in ((self.k, before[0]), (self.v, before[1])):
            for old, new, part in copies:
                b[:, new, :, :part] = b[:, old, :, :part]
            assert torch.equal(c, b)


@pytest.mark.parametrize("n_pages,rows,width,page,pad", [(1, 1, 1, 16, 0), (31, 3, 9, 16, 0), (64, 5, 20, 32, 3), (1000, 40, 30, 64, 0),
                                                         (5000, 700, 7, 128, 1), (40001, 1100, 33, 16, 0), (4097, 1, 4000, 16, 0)])
def test_resize(tpa, n_pages, rows, width, page, pad):
    b = Both(n_pages, rows, width, page, pad=pad)
    r = np.random.default_rng(n_pages)
    lens = [0] * rows
    for step in range(8):
        fill = r.choice([0.3, 0.8])
        for i in range(rows):
            if r.random() < 0.4:
                most = min(width * page, max(1, int(2 * fill * n_pages * page / rows)))
                lens[i] = int(r.integers(0, most + 1)) if r.random() < 0.8 else 0
        b.resize(tpa, lens)
        tpa.sync_status()
        if b.left.item() < 0:  # rows that did not grow have fewer pages than their lengths need: go back to what they hold
            lens = [min(n, len(row) * page) for n, row in zip(lens, b.pool.rows)]
            b.resize(tpa, lens)
    b.resize(tpa, lens)  # nothing changes
    b.resize(tpa, [0] * rows)
    assert b.left.item() == n_pages and not any(b.pool.refs)
    tpa.sync_status()


def test_resize_to_the_last_page(tpa):
    b = Both(100, 4, 60, 16)
    b.resize(tpa, [25 * 16] * 4)
    assert b.left.item() == 0
    b.resize(tpa, [25 * 16 + 1, 25 * 16, 24 * 16, 0])   # what goes back is there for what grows
    b.resize(tpa, [25 * 16 + 1, 60 * 16, 24 * 16, 60 * 16])
    assert b.left.item() < 0
    tpa.sync_status()


def test_most_rows(tpa):
    b = Both(20000, 8192, 3, 16)
    r = np.random.default_rng(2)
    for _ in range(3):
        b.resize(tpa, r.integers(0, 33, 8192).tolist())
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.paged_resize(torch.full((8193, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(8193, dtype=torch.int32, device="cuda"),
                         b.refs, 16)
    tpa.sync_status()


def test_no_rows_counts_the_free_pages(tpa):
    refs = _i32([0, 1, 0, 2, 0]).cuda()
    empty = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    left = tpa.paged_resize(empty, torch.zeros(0, dtype=torch.int32, device="cuda"), refs, 16)
    assert left.item() == 3


@pytest.mark.parametrize("layers,hkv,d,page", [(1, 1, 64, 16), (3, 2, 128, 64), (2, 5, 64, 128), (1, 8, 128, 32)])
def test_fork(tpa, layers, hkv, d, page):
    b = Both(300, 12, 10, page, layers, hkv, d)
    b.resize(tpa, [0, 3 * page, 5, 2 * page + 1, 4 * page - 1, page] + [0] * 6)
    b.fork(tpa, [1, 2, 3, 3, 4, 0], [6, 7, 8, 9, 10, 11])      # whole pages alone, a part alone, both, nothing
    tpa.sync_status()
    b.fork(tpa, [3, 4, 5], [6, 8, 7])                           # rows that hold pages already
    b.fork(tpa, [3, 4, 5], [6, 8, 7])                           # the same again
    lens = b.lens.tolist()
    lens[6] += page                                             # a fork goes on by itself
    lens[3] = 0                                                 # its source ends; what is shared stays
    b.resize(tpa, lens)
    b.resize(tpa, [0] * 12)
    assert b.left.item() == 300
    tpa.sync_status()


def test_fork_many(tpa):
    b = Both(4000, 500, 12, 16, 2)
    r = np.random.default_rng(5)
    lens = r.integers(0, 190, 60).tolist() + [0] * 440
    b.resize(tpa, lens)
    for _ in range(3):
        dst = (60 + r.permutation(440)[:300]).tolist()
        b.fork(tpa, r.integers(0, 60, 300).tolist(), dst)
    tpa.sync_status()


def test_fork_without_room(tpa):
    b = Both(10, 6, 9, 16, 1)
    b.resize(tpa, [7 * 16 + 3, 0, 16, 0, 0, 0])
    b.fork(tpa, [0, 0], [2, 3])       # row 2 gives its page back: two free, two needed
    b.fork(tpa, [0, 0], [4, 5])       # none free: the rows stay empty
    assert b.left.item() == -2 and b.lens.tolist()[4:] == [0, 0]
    tpa.sync_status()
    b.fork(tpa, [0, 0], [2, 4])
    b.fork(tpa, [], [])


def test_forks_that_make_no_sense_are_not_done(tpa):
    b = Both(50, 6, 4, 16, 1)
    b.resize(tpa, [20, 40, 16, 0, 0, 0])
    state = [x.clone() for x in (b.table, b.refs, b.lens, b.k, b.v)]
    for src, dst in (([0, 1], [3, 3]), ([0, 3], [3, 4]), ([0], [0]), ([6], [3]), ([-1], [3]), ([0], [6]), ([0], [-1]),
                     ([0, 1], [3, 2 ** 31 - 1])):
        left = tpa.paged_fork(b.k, b.v, b.pages, b.lens, b.refs, _i32(src).cuda(), _i32(dst).cuda())
        assert left.item() == -2 ** 31
        with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
            tpa.sync_status()
        assert all(torch.equal(x, y) for x, y in zip(state, (b.table, b.refs, b.lens, b.k, b.v)))
    for bad in (-1, 4 * 16 + 1):
        b.lens[1] = bad
        left = tpa.paged_fork(b.k, b.v, b.pages, b.lens, b.refs, _i32([0, 1]).cuda(), _i32([3, 4]).cuda())
        assert left.item() == -2 ** 31
        with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
            tpa.sync_status()
        assert torch.equal(b.table, state[0]) and torch.equal(b.refs, state[1])


def test_broken_state_is_reported_and_not_followed(tpa):
    b = Both(20, 3, 4, 16, 1)
    b.resize(tpa, [40, 20, 0])
    for lens in ([-1, 20, 0], [65, 20, 0], [2 ** 31 - 1, 20, 0], [-2 ** 31, 20, 0]):  # of row 0: it stays as it is
        before = b.table.clone()
        b.lens.copy_(_i32(lens))
        left = tpa.paged_resize(b.pages, b.lens, b.refs, 16)
        with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
            tpa.sync_status()
        assert torch.equal(b.table, before) and left.item() == 15
    b.lens.copy_(_i32([0, 20, 0]))
    b.pages[0, 1] = 20                     # no such page
    b.refs[b.pages[0, 2].item()] = 0       # not in use
    refs = b.refs.clone()
    first = b.pages[0, 0].item()
    tpa.paged_resize(b.pages, b.lens, b.refs, 16)
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()
    refs[first] -= 1
    assert torch.equal(b.refs, refs) and (b.pages[0] == -1).all()


def test_fork_past_32_bits(tpa):
    """Layers and pages whose bytes pass 2^32."""
    n_pages = 70000
    k = torch.zeros((3, n_pages, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    pages = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    pages[0, 0], pages[0, 1] = 5, n_pages - 1
    refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
    refs[n_pages - 3] = 0
    lens = _i32([16 + 9, 0]).cuda()
    for layer in range(3):
        k[layer, n_pages - 1] = layer + 1
        v[layer, n_pages - 1] = -layer - 1
    left = tpa.paged_fork(k, v, pages, lens, refs, _i32([0]).cuda(), _i32([1]).cuda())
    tpa.sync_status()
    assert left.item() == 0 and pages.tolist() == [[5, n_pages - 1, -1], [5, n_pages - 3, -1]] and lens.tolist() == [25, 25]
    for layer in range(3):
        assert (k[layer, n_pages - 3, :, :9] == layer + 1).all() and (k[layer, n_pages - 3, :, 9:] == 0).all()
        assert (v[layer, n_pages - 3, :, :9] == -layer - 1).all() and (v[layer, n_pages - 3, :, 9:] == 0).all()


def test_captured_between_batches(tpa):
    """Sequences end, new ones come and fork, in one captured step that is replayed with other lengths."""
    b = Both(200, 12, 8, 16, 2)
    src, dst = _i32([4, 4, 5, 5]).cuda(), _i32([6, 7, 8, 9]).cuda()
    wanted = torch.zeros(12, dtype=torch.int32, device="cuda")
    b.resize(tpa, [0] * 12)
    graph = torch.cuda.CUDAGraph()

    def step():
        b.lens.copy_(wanted)
        room = tpa.paged_resize(b.pages, b.lens, b.refs, 16)
        return room, tpa.paged_fork(b.k, b.v, b.pages, b.lens, b.refs, src, dst)

    with torch.cuda.graph(graph):
        room, left = step()
    r = np.random.default_rng(3)
    for _ in range(5):
        lens = r.integers(0, 100, 6).tolist() + [0] * 6
        before = b.k.clone(), b.v.clone()
        wanted.copy_(_i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert room.item() == b.pool.resize(lens)
        n, copies = b.pool.fork([4, 4, 5, 5], [6, 7, 8, 9])
        b.left.copy_(left)
        b.check(n)
        for c, x in ((b.k, before[0]), (b.v, before[1])):
            for old, new, part in copies:
                x[:, new, :, :part] = x[:, old, :, :part]
            assert torch.equal(c, x)
    tpa.sync_status()


def test_forked_samples_go_on_apart(tpa):
    """A prompt's forks append tokens of their own: attention of each sample is that over its own history."""
    from oracle.paged import attend_sequence
    hq, hkv, d, page = 4, 2, 64, 16
    b = Both(40, 4, 6, page, 1, hkv, d)
    g = torch.Generator().manual_seed(9)
    rand = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    b.resize(tpa, [37, 0, 0, 0])
    offsets = _i32([0, 37, 37, 37, 37]).cuda()
    k, v = rand(37, hkv, d), rand(37, hkv, d)
    tpa.paged_append(b.k[0], b.v[0], b.pages, offsets, b.lens, k, v)
    b.fork(tpa, [0, 0, 0], [1, 2, 3])
    history = [[k, v] for _ in range(4)]
    for n in (1, 14, 3):
        b.resize(tpa, [x + n for x in b.lens.tolist()])
        offsets = _i32([n * i for i in range(5)]).cuda()
        q, k, v = rand(4 * n, hq, d), rand(4 * n, hkv, d), rand(4 * n, hkv, d)
        tpa.paged_append(b.k[0], b.v[0], b.pages, offsets, b.lens, k, v)
        o, _ = tpa.paged_attn_fwd(b.k[0], b.v[0], b.pages, offsets, b.lens, q, max_q_len=n)
        for s in range(4):
            rows = slice(n * s, n * s + n)
            history[s] = [torch.cat([h, x[rows]]) for h, x in zip(history[s], (k, v))]
            ref, _, size = attend_sequence(q[rows].cpu(), history[s][0].cpu(), history[s][1].cpu())
            off = (o[rows].double().cpu() - ref).abs() - ((2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * ref.abs())
            assert off.max() <= 0
    tpa.sync_status()
