"""Attention over page tables and lengths that the calls just before it write: those kernels may still run when the
attention's starts.  Results are those of the same calls with a wait after each, bit for bit."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE, WIDTH, HKV, D = 16, 48, 2, 64


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Case:
    def __init__(self, S, n, seed):
        g = torch.Generator().manual_seed(seed)
        r = np.random.default_rng(seed)
        rand = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        self.S, self.n = S, n
        n_pages = 4 * S * WIDTH
        self.start = rand(n_pages, HKV, PAGE, D), rand(n_pages, HKV, PAGE, D)
        self.k, self.v = (x.clone() for x in self.start)
        self.q = rand(S * n, 4 * HKV, D)
        self.lens = [r.integers(n, PAGE * WIDTH + 1, S).tolist() for _ in range(3)]
        self.parents = _i32([-1 if i == 0 else int(r.integers(0, i)) for _ in range(S) for i in range(n)])
        self.offsets = _i32([n * s for s in range(S + 1)])
        self.refs = torch.zeros(n_pages, dtype=torch.int32).cuda()
        words = (n + 31) // 32
        self.positions, self.masks = (torch.zeros(s, dtype=torch.int32).cuda() for s in ((S * n,), (S * n, words)))

    def attend(self, tpa, pages, lens, wait, workspace, tree):
        tpa.draft_masks(self.parents, self.offsets, lens, self.n, out=(self.positions, self.masks))
        wait()
        args = self.k, self.v, pages, self.offsets, lens, self.q
        if tree:
            out = tpa.paged_attn_tree_fwd(*args, self.masks, self.n, workspace=workspace)
        else:
            out = tpa.paged_attn_fwd(*args, self.n, workspace=workspace)
        wait()
        return out

    def put_back(self):
        for x, y in zip((self.k, self.v), self.start):
            x.copy_(y)
        self.refs.zero_()


def _resized(tpa, c, wait, workspace, tree):
    """The rows' pages given back and handed out again for other lengths, over and over."""
    pages, lens = torch.full((c.S, WIDTH), -1, dtype=torch.int32).cuda(), [_i32(x) for x in c.lens]
    free = _i32([0])
    out = []
    for i in range(24):
        tpa.paged_resize(pages, lens[i % 3], c.refs, PAGE, out=free)
        wait()
        out += c.attend(tpa, pages, lens[i % 3], wait, workspace, tree)
    return out


def _forked(tpa, c, wait, workspace, tree):
    """The rows made copies of one group of others and then of the other, tables and lengths."""
    S = c.S
    pages, lens = torch.full((3 * S, WIDTH), -1, dtype=torch.int32).cuda(), _i32(c.lens[0] + c.lens[1] + [0] * S)
    free = _i32([0])
    assert tpa.paged_resize(pages, lens, c.refs, PAGE).item() > 0
    src, dst = [_i32(range(S)), _i32(range(S, 2 * S))], _i32(range(2 * S, 3 * S))
    out = []
    for i in range(24):
        tpa.paged_fork(c.k, c.v, pages, lens, c.refs, src[i % 2], dst, out=free)
        wait()
        out += c.attend(tpa, pages[2 * S:], lens[2 * S:], wait, workspace, tree)
    return out


def _moved_on(tpa, c, wait, workspace, tree):
    """Lengths and keys that the compacted cache leaves: each step takes the first of the new tokens out."""
    S, n = c.S, c.n
    pages = _i32([[s * WIDTH + j for j in range(WIDTH)] for s in range(S)])
    lens = [_i32([max(n + 24, x) for x in c.lens[0]]), _i32([0] * S)]
    path, count = _i32([list(range(1, n))] * S), _i32([n - 1] * S)
    out = []
    for i in range(24):
        tpa.paged_compact(c.k, c.v, pages, c.offsets, lens[i % 2], path, count, out=lens[(i + 1) % 2])
        wait()
        out += c.attend(tpa, pages, lens[(i + 1) % 2], wait, workspace, tree)
    return out


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("calls", [_resized, _forked, _moved_on])
@pytest.mark.parametrize("S,n", [(5, 4), (100, 4), (40, 40)])
def test_attention_right_behind_the_calls_that_write_its_tables(tpa, S, n, calls, tree):
    c = Case(S, n, S + n)
    workspace = torch.empty(tpa.paged_attn_workspace_bytes(n, 4 * HKV, HKV, D), dtype=torch.uint8, device="cuda")
    want = calls(tpa, c, torch.cuda.synchronize, workspace, tree)
    for _ in range(4):
        c.put_back()
        got = calls(tpa, c, lambda: None, workspace, tree)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    tpa.sync_status()
