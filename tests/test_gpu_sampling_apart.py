"""The sampling operators where calls meet: on another stream, from two streams at once, from two
threads, in a graph beside another one; and inputs at the ends of what they allow.  All results are equal to those of
the calls made one after another."""
import threading

import pytest
import torch

from oracle.draft import accept

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


class Round:
    """A cache of 2 S sequences, half of them forks of the others, and a step's inputs; `run` makes all calls and returns what they give and what they leave."""

    def __init__(self, seed, n, d=64, page=16, S=5, hq=8, hkv=2, vocab=999, window=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.S, self.window, width = n, S, window, 40
        rand = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        self.k, self.v = rand(2, 3 * S * width, hkv, page, d), rand(2, 3 * S * width, hkv, page, d)
        self.refs = torch.zeros(3 * S * width, dtype=torch.int32).cuda()
        self.pages = torch.full((2 * S, width), -1, dtype=torch.int32).cuda()
        kv = torch.randint(1, width * page // 2, (S,), generator=g)
        self.lens = torch.cat([kv, torch.zeros(S, dtype=torch.int64)]).to(torch.int32).cuda()
        self.src, self.dst = _i32(range(S)).cuda(), _i32(range(S, 2 * S)).cuda()
        self.offsets = _i32([n * i for i in range(2 * S + 1)]).cuda()
        rows = 2 * S * n
        self.parents = _i32([-1 if i == 0 else int(torch.randint(0, i, (1,), generator=g)) for _ in range(2 * S) for i in range(n)]).cuda()
        self.q, self.logits, self.u = rand(rows, hq, d), rand(rows, vocab), torch.rand(rows, generator=g).cuda()
        self.drafted = torch.randint(0, 4, (rows,), generator=g).to(torch.int32).cuda()
        self.logits[:, 4:] = -float("inf")

    def state(self):
        return [x.clone() for x in (self.k, self.v, self.refs, self.pages, self.lens)]

    def put_back(self, state):
        for x, y in zip((self.k, self.v, self.refs, self.pages, self.lens), state):
            x.copy_(y)

    def run(self, tpa, stream=None):
        """The prompts' pages, their forks, pages for the drafts of all (a sequence's own: it writes there), and a step."""
        n = self.n
        free = tpa.paged_resize(self.pages, self.lens, self.refs, self.k.shape[3], stream=stream)
        free2 = tpa.paged_fork(self.k, self.v, self.pages, self.lens, self.refs, self.src, self.dst, stream=stream)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            self.lens += n
        free3 = tpa.paged_resize(self.pages, self.lens, self.refs, self.k.shape[3], stream=stream)
        positions, masks = tpa.draft_masks(self.parents, self.offsets, self.lens, n, self.window, stream=stream)
        o, lse = tpa.paged_attn_tree_fwd(self.k[0], self.v[0], self.pages, self.offsets, self.lens, self.q, masks, n, positions,
                                         window=self.window, stream=stream)
        sampled, logp = tpa.sample_tokens(self.logits, self.u, 0.9, 3, 0.95, 0.001, stream=stream)
        plain, plain_logp = tpa.sample_tokens(self.logits, self.u, 0.9, stream=stream)
        tokens, path, count = tpa.accept_drafts(self.parents, self.offsets, self.drafted, sampled, n, stream=stream)
        lens = tpa.paged_compact(self.k, self.v, self.pages, self.offsets, self.lens, path, count, stream=stream)
        return [free, free2, free3, positions, masks, o, lse, sampled, logp, plain, plain_logp, tokens, path, count, lens]


def _same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("n,window", [(1, 0), (16, 0), (7, 20), (64, 0), (40, 100)])
def test_on_another_stream(tpa, n, window):
    r = Round(n, n, window=window)
    start = r.state()
    want = r.run(tpa)
    left = r.state()
    r.put_back(start)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = r.run(tpa, stream=side)
    side.synchronize()
    _same(want, got)
    _same(left, r.state())
    assert int(want[13].max()) > 1 or n == 1  # something was accepted
    tpa.sync_status()


def test_two_streams_at_once(tpa):
    rounds = [Round(100 + i, n, d, S=S) for i, (n, d, S) in enumerate([(16, 64, 8), (48, 128, 20)])]
    starts = [r.state() for r in rounds]
    want = [r.run(tpa) for r in rounds]
    left = [r.state() for r in rounds]
    sides = [torch.cuda.Stream() for _ in rounds]
    for _ in range(10):
        for r, s in zip(rounds, starts):
            r.put_back(s)
        torch.cuda.synchronize()
        got = [r.run(tpa, stream=s) for r, s in zip(rounds, sides)]
        torch.cuda.synchronize()
        for i in range(2):
            _same(want[i], got[i])
            _same(left[i], rounds[i].state())
    tpa.sync_status()


def test_two_graphs_replayed_at_once(tpa):
    rounds = [Round(200 + i, n, d, S=S) for i, (n, d, S) in enumerate([(16, 128, 8), (48, 64, 20)])]
    starts = [r.state() for r in rounds]
    want = [r.run(tpa) for r in rounds]
    left = [r.state() for r in rounds]
    graphs, got = [], []
    for r, s in zip(rounds, starts):
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(r.run(tpa))
    sides = [torch.cuda.Stream() for _ in rounds]
    for _ in range(10):
        for r, s in zip(rounds, starts):
            r.put_back(s)
        torch.cuda.synchronize()
        for graph, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            _same(want[i], got[i])
            _same(left[i], rounds[i].state())
    tpa.sync_status()


def test_pools_of_different_sizes_from_two_threads(tpa):
    # (their kernels want different amounts of shared memory)
    failed = []

    def work(rows, n_pages):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                pages, refs = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda"), torch.zeros(n_pages, dtype=torch.int32, device="cuda")
                for i in range(60):
                    lens = torch.full((rows,), 16 * (i % 3), dtype=torch.int32, device="cuda")
                    left = tpa.paged_resize(pages, lens, refs, 16)
                    if left.item() != n_pages - rows * (i % 3):
                        failed.append((rows, i, left.item()))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in ((1, 100), (7000, 20000), (8192, 1 << 23), (6500, 14000))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    tpa.sync_status()


def test_more_pages_wanted_than_32_bits_count(tpa):
    width, rows = (1 << 26) - 1, 33   # 33 (2^26 - 1) pages: past 2^31
    refs = torch.zeros(50, dtype=torch.int32, device="cuda")
    pages = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    lens[3] = 40
    assert tpa.paged_resize(pages, lens, refs, 16).item() == 47
    lens.fill_(16 * width)
    left = tpa.paged_resize(pages, lens, refs, 16).item()
    assert left == -2 ** 31 + 1       # (as many as are told)
    assert refs.tolist() == [1] * 3 + [0] * 47
    assert pages[3, :4].tolist() == [0, 1, 2, -1] and int((pages >= 0).sum()) == 3
    lens[5:] = 0
    assert tpa.paged_resize(pages, lens, refs, 16).item() == 47 - (5 * width - 3)
    lens.zero_()
    assert tpa.paged_resize(pages, lens, refs, 16).item() == 50
    tpa.sync_status()


def test_negative_tokens_are_nobodys(tpa):
    # a tree padded with -1, and a row with nothing to draw
    parents, drafted, sampled = [-1, 0, 0, 1], [7, -1, 5, 6], [-1, 6, 0, 0]
    args = [_i32(x).cuda() for x in (parents, [0, 4], drafted, sampled)]
    tokens, path, count = tpa.accept_drafts(*args, 4)
    want = accept(parents, drafted, sampled, 4)
    assert want == ([0], [-1])
    assert path.tolist() == [[0, -1, -1, -1]] and tokens.tolist() == [[-1] * 4] and count.tolist() == [1]
    tpa.sync_status()


def test_same_logits_in_many_rows_and_odd_strides(tpa):
    # rows of a wider matrix, each beginning off a 16-byte border; a row's result is that of the row alone
    g = torch.Generator().manual_seed(5)
    wide = torch.randn((9, 5003), generator=g).to(torch.bfloat16).cuda()
    for at in range(1, 8):
        x, u = wide[:, at:at + 4987], torch.rand(9, generator=g).cuda()
        t, l = tpa.sample_tokens(x, u, 0.8, 40, 0.9)
        for i in range(9):
            t1, l1 = tpa.sample_tokens(x[i:i + 1].clone(), u[i:i + 1], 0.8, 40, 0.9)
            assert t1[0] == t[i] and l1[0] == l[i]
    tpa.sync_status()


def _steps(tpa, r, sampled, steps, wait):
    """Steps that each take the one before's lengths, in the same memory over and over."""
    n, S = r.n, 2 * r.S
    new = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, positions, masks = [r.lens.clone(), new(S)], new(S * n), new(S * n, 1)
    tokens, path, count = new(S, n), new(S, n), new(S)
    for i in range(steps):
        tpa.draft_masks(r.parents, r.offsets, lens[i % 2], n, out=(positions, masks))
        if wait:
            torch.cuda.synchronize()
        tpa.accept_drafts(r.parents, r.offsets, r.drafted, sampled[i % len(sampled)], n, out=(tokens, path, count))
        if wait:
            torch.cuda.synchronize()
        tpa.paged_compact(r.k, r.v, r.pages, r.offsets, lens[i % 2], path, count, out=lens[(i + 1) % 2])
        if wait:
            torch.cuda.synchronize()
    return [*lens, positions, masks, tokens, path, count, r.k.clone(), r.v.clone()]


def test_a_stream_of_calls_without_waiting(tpa):
    r = Round(300, 16)
    tpa.paged_resize(r.pages, r.lens.fill_(600), r.refs, 16)  # (10 rows of 38 pages, of 600)
    sampled = [tpa.sample_tokens(r.logits, torch.rand_like(r.u), 0.9)[0] for _ in range(3)]
    start = r.state()
    want = _steps(tpa, r, sampled, 30, True)
    assert not torch.equal(r.k, start[0])
    assert int(want[0].min()) > 16
    for _ in range(5):
        r.put_back(start)
        _same(want, _steps(tpa, r, sampled, 30, False))
    graph = torch.cuda.CUDAGraph()
    r.put_back(start)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = _steps(tpa, r, sampled, 30, False)
    for _ in range(3):
        r.put_back(start)
        graph.replay()
        torch.cuda.synchronize()
        _same(want, got)
    tpa.sync_status()
