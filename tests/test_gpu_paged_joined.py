"""Paged attention where tiles of one batch are cut into very different numbers of parts: every row of each is joined, for
chains and trees.  Bounds as in test_gpu_tree_drafts.py."""
import pytest
import torch

from oracle.draft import attend_tree
from _paged import Batch
from _pipeline import check_guards, guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,d,page", [
    ([1], [20001], 16, 2, 128, 64),                              # 79 parts of 8 rows
    ([48], [9000], 16, 2, 128, 64),                              # 36 of 256 and of 128 rows
    ([2, 1, 2], [9000, 7, 300], 8, 1, 64, 16),                   # few rows: many parts beside none
    ([40, 1, 3, 2], [12000, 50, 300, 2500], 16, 2, 128, 128),    # many rows: many parts beside few and none
    ([100, 2, 2, 33], [3000, 6000, 10, 33], 8, 2, 64, 32),
    ([17] * 9 + [1], [700] * 9 + [9000], 6, 2, 128, 32),
    ([300], [4000], 8, 1, 64, 64),
    ([4] * 40, [260] * 40, 8, 2, 128, 16),                       # two parts at most
])
@pytest.mark.parametrize("tree", [False, True])
def test_every_row_is_joined(tpa, q_lens, kv_lens, hq, hkv, d, page, tree):
    b = Batch(q_lens, kv_lens, hq, hkv, d, page, seed=len(q_lens) + d)
    bo, o = guarded(b.q.shape, torch.bfloat16)
    bl, lse = guarded(b.q.shape[:2], torch.float32)
    o.fill_(777.0)
    lse.fill_(777.0)
    most = max(q_lens)
    parents = [-1 if i == 0 else (i - 1 if not tree else (i - 1) // 2) for n in q_lens for i in range(n)]
    if tree:
        positions, masks = tpa.draft_masks(torch.tensor(parents, dtype=torch.int32).cuda(), b.offsets, b.kv_lens, most)
        tpa.paged_attn_tree_fwd(*b.cache, b.q, masks, most, out=o, lse=lse)
    else:
        tpa.paged_attn_fwd(*b.cache, b.q, most, out=o, lse=lse)
    tpa.sync_status()
    check_guards(bo, "o")
    check_guards(bl, "lse")
    assert (o != 777.0).all() and (lse != 777.0).all()
    at = 0
    for s, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        seen = torch.ones((n, kv), dtype=torch.bool)
        seen[:, kv - n:] = False
        for i in range(n):
            up = i
            while up >= 0:
                seen[i, kv - n + up] = True
                up = parents[at + up]
        ref, rl, size = attend_tree(b.q[at:at + n].cpu(), b.sequence(s, b.k_cache), b.sequence(s, b.v_cache), seen)
        got, gl = o[at:at + n].double().cpu(), lse[at:at + n].double().cpu()
        assert ((got - ref).abs() <= (2.0 ** -8 + 2.0 ** -14) * size + 2.0 ** -8 * ref.abs()).all(), f"sequence {s}"
        assert ((gl - rl).abs() <= 2.0 ** -14 + 2.0 ** -23 * rl.abs()).all(), f"sequence {s}: LSE"
        at += n
