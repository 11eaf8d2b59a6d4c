"""Drafted trees whose description is broken: what is reported, and what the others' results are beside it."""
import pytest
import torch

from oracle.draft import accept, masks as oracle_masks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("bad", [-1, -5, -2 ** 31])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_negative_lengths_are_reported(tpa, at, bad):
    # as the attention reports them; (sequence 1 has no new tokens)
    trees, lens = [[-1, 0, 0, 1], [], [-1, 0, 1]], [10, 7, 2]
    lens[at] = bad
    positions, masks = torch.full((7,), 77, dtype=torch.int32, device="cuda"), torch.full((7, 1), 77, dtype=torch.int32, device="cuda")
    tpa.draft_masks(_i32([p for t in trees for p in t]), _i32([0, 4, 4, 7]), _i32(lens), 4, out=(positions, masks))
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()
    row = 0
    for t, n in zip(trees, lens):
        want = oracle_masks(t, n - len(t), 1) if n >= 0 else ([77] * len(t), [[77]] * len(t))
        assert positions[row:row + len(t)].tolist() == want[0] and masks[row:row + len(t)].tolist() == want[1]
        row += len(t)
    tpa.sync_status()


@pytest.mark.parametrize("at,bad", [(0, 0), (1, 1), (2, 3), (5, -2), (3, 2 ** 31 - 1), (7, -2 ** 31), (4, 4), (6, 6)])
def test_tokens_with_broken_parents_are_not_accepted(tpa, at, bad):
    # every token fits; the broken one is nobody's child (a sequence's row 0 stands whatever its parent)
    trees = [[-1, 0, 1, 2], [-1, 0, 1, 2]]
    parents = trees[0] + trees[1]
    parents[at] = bad
    x = torch.zeros(8, dtype=torch.int32, device="cuda")
    tokens, path, count = tpa.accept_drafts(_i32(parents), _i32([0, 4, 8]), x, x, 4)
    with pytest.raises(tpa.TpaError, match="INVALID_ARG"):
        tpa.sync_status()
    trees[at // 4][at % 4] = -1
    for s, t in enumerate(trees):
        rows, out = accept(t, [0] * 4, [0] * 4, 4)
        assert count[s] == len(rows) and path[s].tolist() == rows + [-1] * (4 - len(rows))
        assert tokens[s].tolist() == out + [-1] * (4 - len(rows))
    tpa.sync_status()
