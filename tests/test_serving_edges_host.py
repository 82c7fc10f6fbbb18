"""Rules of the serving step's sources and documents that no run shows (no GPU)."""
import ast
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_decode_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_launch_that_begins_before_its_wait_reads_past_l1():
    """The state's launch of a plan or release reads, before any wait of its own, what the call before has written in place."""
    code = source("pages.cu")
    for name in ("past", "news", "ended"):
        assert not re.search(r"\ba\.%s\[" % name, code), f"{name} is read through L1"
    assert not re.search(r"\*a\.n_free\b(?!_out)", code), "n_free is read through L1"
    assert re.search(r"T read\(const PagesArgs& a, const T\* p\) \{\s*return a\.parts == PAGES_STATE \? __ldcg\(p\) : \*p;", code)
    for kernel in ("plan_pages_kernel", "release_pages_kernel"):
        before = code[code.index(f"__launch_bounds__(PG_THREADS) {kernel}"):]
        before = before[:before.index("PAGES_STATE) {")]
        assert before.count("read(a, a.past + b)") == 1
        assert "a.shares[" not in before and "a.table" not in before and "a.free_pages" not in before, kernel


def test_the_readme_keeps_the_shared_pages():
    """Its serving step plans with shared pages, so the release before it must leave them where they are."""
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    steps = [ast.parse(b) for b in blocks if "moe.release_pages(" in b and "moe.plan_pages(" in b]
    assert steps
    for step in steps:
        calls = {n.func.attr: {k.arg for k in n.keywords} for n in ast.walk(step)
                 if isinstance(n, ast.Call) and isinstance(n.func, ast.Attribute)}
        if "shared_pages" in calls["plan_pages"]:
            assert "shared" in calls["release_pages"], "the prefix's pages would go to the free stack"
            for name in ("release_pages", "plan_pages", "shared_prefix_attention"):
                assert ("shares" in calls[name]) == ("shares" in calls["plan_pages"]), "the same sequences share in all calls"
