"""tpa_sync_status gathers the status words of all kernels in one read, and
reports and clears each of them."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpa():
    import prefix_shared_tree_attention_gb300 as tpa
    tpa.lib()
    tpa.device_check()
    return tpa


def test_no_dearer_than_a_few_copies(tpa):
    """The words of nine translation units: a copy for each takes 83 us, one of all of them behind a kernel that
    gathers them 20, and the read of a tensor's one value 10."""
    value = torch.zeros(1, dtype=torch.int32, device="cuda")

    def least(call):
        call()
        times = []
        for _ in range(200):
            start = time.perf_counter()
            call()
            times.append(time.perf_counter() - start)
        return min(times)

    assert least(tpa.sync_status) <= 4 * least(value.item)


def test_words_of_several_kernels_at_once(tpa):
    table = tpa.rope_table(8, 64)
    x = torch.zeros((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    p = torch.full((1, 2, 16), 1.0, device="cuda")
    u, un = torch.zeros((1, 1), device="cuda"), torch.zeros(1, device="cuda")

    def rope():  # positions past the table
        tpa.qk_norm_rope_fwd(torch.full((4,), 8, dtype=torch.int32, device="cuda"), x, x.clone(), table)

    def verify():  # a token outside the vocabulary
        tpa.verify_drafts(p, torch.full((1, 1), 16, dtype=torch.int32, device="cuda"), u, un)

    for calls, status in (((rope,), "INVALID_ARG"), ((verify,), "INVALID_ARG"), ((rope, verify), "INVALID_ARG"),
                          ((lambda: tpa.wait_probe(1000, False),), "DEVICE_TIMEOUT")):
        for call in calls:
            call()
        with pytest.raises(tpa.TpaError, match=status):
            tpa.sync_status()
        tpa.sync_status()


def test_on_a_stream_of_its_own(tpa):
    side = torch.cuda.Stream()
    tpa.wait_probe(1000, False, stream=side)
    with pytest.raises(tpa.TpaError, match="DEVICE_TIMEOUT"):
        tpa.sync_status(stream=side)
    tpa.sync_status(stream=side)
    tpa.sync_status()
