"""Draws from vocabularies far beyond a model's: the sums keep what
tpa_verify_drafts promises, 2^-41 + vocab 2^-56 of the whole."""
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


@pytest.mark.parametrize("odd", [0, 1])  # rows that are read by 16 bytes, and by 4
def test_the_sums_of_a_long_row(tpa, odd):
    """One half of the row is 0.6, whose running sums round, the other 1/2, whose sums are exact, so that an error of the
    first half moves the draw in the second.  The token follows from whole numbers.  A draw is asked for in the middle
    of an entry: the sums may be off by 2^-29 + 2^-41 of 2^26.2, 0.14, or 0.29 of an entry."""
    V = (1 << 27) + odd
    half = V // 2
    row = torch.full((V,), 0.5, device="cuda")
    row[:half] = 0.6
    c = Fraction(float(torch.tensor(0.6)))
    total = half * c + Fraction(V - half, 2)
    p = torch.zeros((V + odd), device="cuda")[odd:]
    p.copy_(row)
    none = torch.zeros((1, 0), device="cuda")
    toks = none.to(torch.int32)
    tried = 0
    g = torch.Generator().manual_seed(3)
    while tried < 8:
        u = (0.56 + 0.4 * torch.rand(1, generator=g)).float()
        at = Fraction(float(u)) * total - half * c  # of the second half
        if at <= 0 or not Fraction(3, 10) <= (at * 2) % 1 <= Fraction(7, 10):
            continue
        tried += 1
        tokens, n = tpa.verify_drafts(p.view(1, 1, V), toks, none, u.cuda())
        assert int(n[0]) == 0 and int(tokens[0, 0]) == half + int(at * 2), float(u)
    tpa.sync_status()
