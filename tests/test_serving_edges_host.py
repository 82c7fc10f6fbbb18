"""Rules of the serving step's sources and documents that no run shows (no GPU)."""
import ast
import math
import os
import re

import numpy as np

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


def test_the_softmax_scores_error_is_a_bound():
    """In units of 2^-24, relative to the largest possible score 1 / total: exp2 within 2 units in the last place; its argument
    from a difference and a product (a unit each) by a constant that is itself off; the sum's terms have the same errors, the
    exponents' weighted by the scores; its additions are a lane's (32 of 1024 experts) and five steps; a reciprocal and a
    product."""
    unit, exp2 = 2.0 ** -24, 4.0
    off = abs(float(np.float32(1.44269504)) / math.log2(math.e) - 1) / unit
    argument = 2 + off
    d = np.linspace(0, 40, 400001)
    score_times = (np.exp(-d) * d).max()                     # of one expert, d below the largest
    rest = 1023 * np.exp(-d)
    mean = (rest * d / (1 + rest)).max()                     # sum p |x - m|: largest where all but one are equally far
    rng = np.random.default_rng(1)
    for _ in range(200):
        x = -rng.gamma(rng.uniform(0.1, 8), rng.uniform(0.1, 8), 1024)
        p = np.exp(x - x.max())
        assert (p * (x.max() - x)).sum() / p.sum() <= mean
    bound = exp2 + argument * score_times + exp2 + argument * mean + (32 + 5) + 2
    held = re.search(r"softmax \? (0x[0-9a-f]+)p-24f / total", source("router_grouped.cu")).group(1)
    assert bound <= int(held, 16), (bound, held)


def test_the_binding_allocates_by_torchs_operator_alone():
    code = source("binding.cpp")
    assert "at::detail" not in code and "at::empty(" in code
