"""The counters under profiles/ of the sampling step's operators are those of the
kernels in the tree: each source that they were taken from is named with its
sha256 prefix."""
import hashlib
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = "prefix_shared_tree_attention_gb300/csrc/"


def test_sampling_profiles_match_the_kernel_sources():
    with open(os.path.join(ROOT, "profiles", "sampling_operators_ncu.md")) as f:
        text = f.read()
    named = dict(re.findall(r"^Source: `([^`]+)` sha256 prefix ([0-9a-f]{16})$", text, re.M))
    files = ("sample.cu", "draft.cu", "pages.cu", "paged_few.cu", "paged_tile.cu", "paged_common.cuh")
    assert set(named) == {CSRC + f for f in files}
    for path, prefix in named.items():
        with open(os.path.join(ROOT, path), "rb") as f:
            source = f.read()
        assert hashlib.sha256(source).hexdigest().startswith(prefix), path
        for kernel in re.findall(r"__global__[^;{]*?\b(\w+_kernel)\(", source.decode()):
            assert f"| `{kernel}" in text, kernel
