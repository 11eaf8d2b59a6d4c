"""Batches over a paged cache: a sequence's results are its own whatever stands
in the rows beside it."""
import pytest
import torch

from _paged import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _rising_keys(b, step):
    """Key dimension 0 rises along each sequence; every query's dimension 0 is 0."""
    b.q[..., 0] = 0
    for s, n in enumerate(b.kv_lens_list):
        j = torch.arange(n)
        page = torch.tensor(b.rows[s])[j // b.page]
        b.k_cache[page.cuda(), :, (j % b.page).cuda(), 0] = (j * step).to(torch.bfloat16).cuda()[:, None]


@pytest.mark.parametrize("q_len,hq,hkv,d", [(1, 4, 1, 128), (1, 32, 8, 128), (3, 4, 2, 64), (5, 16, 4, 128), (2, 12, 1, 64),
                                            (7, 3, 1, 128), (2, 17, 1, 64), (150, 4, 1, 128)])
@pytest.mark.parametrize("window", [0, 20000])
def test_queries_of_other_rows_do_not_matter(tpa, q_len, hq, hkv, d, window):
    """A tile's load brings the rows behind its own: padding, or the next sequence's.  Queries there whose scores rise
    along the keys, or are not numbers, leave every bit of the sequence's own results."""
    lens = [n // hkv for n in (90000, 70000, 80001)]  # some ten steps of 128 keys for every CTA
    b = Batch([q_len] * 3, lens, hq, hkv, d, 16, seed=41, extra=40)
    _rising_keys(b, 1.0)
    n = b.total

    def run():
        return [x.clone() for x in tpa.paged_attn_fwd(*b.cache, b.q, max_q_len=q_len, window=window)]

    b.q[n:] = 0
    want = run()
    for fill in (8.0, -8.0, 3e38, float("inf"), float("-inf"), float("nan")):
        b.q[n:] = 0
        b.q[n:, :, 0] = fill
        assert all(torch.equal(x[:n], y[:n]) for x, y in zip(want, run())), fill
    b.q[n:] = 0
    middle, kept = slice(q_len, 2 * q_len), b.q.clone()
    others = [i for i in range(n) if not q_len <= i < 2 * q_len]
    for fill in (8.0, -8.0, 3e38, float("inf"), float("nan")):
        b.q.copy_(kept)
        b.q[middle, :, 0] = fill
        assert all(torch.equal(x[others], y[others]) for x, y in zip(want, run())), fill
    tpa.sync_status()
