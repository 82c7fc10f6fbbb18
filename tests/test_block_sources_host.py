"""Source rules of the decode block's kernels that no run can show (no GPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_decode_gb300", "csrc")


@pytest.mark.parametrize("name", ["attention.cu", "rope.cu", "norm.cu", "matvec4.cu"])
def test_programmatic_dependents_read_by_ordinary_loads(name):
    """These kernels may be resident while the kernel before writes their inputs; the non-coherent path asks for
    memory that is read-only as long as a kernel lasts."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "after_previous()" in code
    for word in ("__ldg", "ld_cached_128", ".nc.", "__restrict__", "ld_stream", "ld_weights"):
        assert word not in code, f"{name} reads through {word}"
