"""Source rules of the serving step's kernels that no run can show (no GPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_decode_gb300", "csrc")


@pytest.mark.parametrize("name", ["prefix_attention.cu", "router_grouped.cu", "pages.cu"])
def test_programmatic_dependents_read_by_ordinary_loads(name):
    """As for the block's kernels: they may be resident while the kernel before writes their inputs."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "after_previous()" in code
    for word in ("__ldg(", "ld_cached_128", ".nc.", "__restrict__", "ld_stream", "ld_weights"):
        assert word not in code, f"{name} reads through {word}"


@pytest.mark.parametrize("name", ["prefix_attention.cu", "router_grouped.cu", "pages.cu"])
def test_no_exchange_behind_a_short_circuit(name):
    """An exchange of a warp that only some of its lanes come to waits for ever: none stands behind && or || or in a branch of
    ?:, but for votes whose other operand is the same in all lanes (named here)."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    found = re.findall(r"(?:&&|\|\||\?)\s*\(?\s*__(?:shfl|any|all|ballot|reduce)\w*\([^;]*;", code)
    uniform = ("ok && __all_sync", "ok = ok && __all_sync")
    for hit in found:
        before = code[max(0, code.index(hit) - 12):code.index(hit)] + hit
        assert any(u in before for u in uniform) or "(__ballot_sync(FULL_MASK, close) >> k & 1u)" in hit, f"{name}: {hit[:120]}"
