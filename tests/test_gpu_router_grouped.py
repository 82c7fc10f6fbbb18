"""moe_router_grouped_topk against its definition in 64 bits.

Ids must be equal: keys are compared as real numbers.  Weights: expf within 2
units (2^-22), a sum of up to 32 terms in five steps, a sum, a quotient and a
product of half a unit each, together below 2^-20; softmax weights that are not
renormalised are divided by a sum of E fast exponentials (2^-22 each, and
|x - m| half units of the exponent, |x - m| weighted by the scores being at
most ln E = 7), together below 2^-18."""
import numpy as np
import pytest
import torch

import mixture_experts_decode_gb300 as moe
import _serving_refs as refs

pytestmark = pytest.mark.gpu


def check(dev, logits, k, bias=None, score="sigmoid", groups=1, top_groups=1, group_score="top2", renorm=True, scale=1.0,
          what=""):
    ids, w = moe.router_grouped_topk(logits.to(dev), k, None if bias is None else bias.to(dev), score, groups, top_groups,
                                     group_score, renorm, scale)
    torch.cuda.synchronize()
    rid, rw = refs.router(logits, k, bias, score, groups, top_groups, group_score, renorm, scale)
    got = ids.cpu().numpy()
    bad = np.nonzero((got != rid).any(1))[0]
    assert not len(bad), f"{what}: {len(bad)} rows of other experts, the first {bad[0]}: {got[bad[0]]} for {rid[bad[0]]}"
    tol = 2.0 ** -18 if score == "softmax" and not renorm else 2.0 ** -20
    np.testing.assert_allclose(w.cpu().numpy().astype(np.float64), rw, rtol=tol, atol=1e-30, err_msg=what)
    return ids, w


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0


def randn(*s, seed=0, std=1.0, dtype=torch.float32):
    return (torch.randn(*s, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top", [(1, 1, 1, 1), (2, 1, 1, 1), (8, 2, 4, 2), (33, 5, 3, 2), (64, 6, 8, 3), (96, 32, 1, 1),
                                            (128, 8, 1, 1), (160, 6, 8, 3), (256, 8, 8, 4), (256, 8, 32, 3), (320, 7, 5, 2),
                                            (512, 12, 16, 16), (1000, 31, 8, 5), (1024, 32, 32, 1)])
def test_shapes(cuda_device, score, E, k, groups, top):
    for group_score in ("max", "top2"):
        for bias in (None, randn(E, seed=E, std=0.1 if score == "sigmoid" else 0.3 / E)):
            for renorm in (True, False):
                check(cuda_device, randn(37, E, seed=E + k), k, bias, score, groups, top, group_score, renorm, 2.5,
                      f"{score} {group_score} bias={bias is not None} renorm={renorm}")


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 300, 20000])
def test_numbers_of_tokens(cuda_device, T):
    check(cuda_device, randn(T, 256, seed=T), 8, randn(256, std=0.1), "sigmoid", 8, 4, "top2", True, 2.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_types_and_strides(cuda_device, dtype):
    for E, pad, at in ((128, 8, 0), (100, 3, 0), (256, 5, 3), (36, 4, 4)):
        base = randn(50, E + pad, seed=E, dtype=dtype)
        on = base.to(cuda_device)[:, at:at + E]
        host = base[:, at:at + E]
        bias = randn(E, std=0.05)
        ids, w = moe.router_grouped_topk(on, 4, bias.to(cuda_device), "sigmoid", 2, 1)
        rid, rw = refs.router(host, 4, bias, "sigmoid", 2, 1, "top2", True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), rid)
        np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=2.0 ** -20)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("near", [2, 9, 20, 31, 60, 256])
@pytest.mark.parametrize("k", [1, 8, 32])
def test_keys_that_fp32_cannot_tell_apart(cuda_device, score, near, k):
    """`near` experts' biases put their keys within 2^-26 of one another, above all others."""
    E, T = 256, 24
    x = randn(1, E, seed=near).expand(T, E).clone()
    x[1:] = x[1:] + 1e-5 * randn(T - 1, E, seed=near + 1)
    p = torch.softmax(x[0].double(), -1) if score == "softmax" else torch.sigmoid(x[0].double())
    bias = torch.full((E,), -2.0, dtype=torch.float64)
    pick = torch.randperm(E, generator=torch.Generator().manual_seed(near))[:near]
    bias[pick] = 1.0 - p[pick]
    check(cuda_device, x, k, bias.float(), score, 1, 1, what=f"{near} near")
    check(cuda_device, x, min(k, 8), bias.float(), score, 8, 3, "top2", what=f"{near} near, groups")


def test_groups_that_fp32_cannot_tell_apart(cuda_device):
    """Every group holds the same two best keys to within 2^-25."""
    E, groups = 64, 8
    x = randn(64, E, seed=3, std=1e-4)
    bias = torch.full((E,), -1.0)
    bias[::8], bias[1::8] = 0.5, 0.25
    for gs in ("top2", "max"):
        check(cuda_device, x, 4, bias, "sigmoid", groups, 3, gs)
    x2 = x.clone()
    x2[:] = x2[:, :8].repeat(1, 8)  # the same values in all groups: the lower groups
    ids, _ = check(cuda_device, x2, 4, bias, "sigmoid", groups, 2, "top2")
    assert bool((ids < 16).all())


def test_equal_keys_go_to_the_lowest_index(cuda_device):
    x = torch.zeros(6, 256)
    x[1, ::2] = 1.0
    x[2] = torch.arange(256) % 3
    x[3] = -0.0
    x[3, 100:] = 0.0
    x[4] = torch.randint(0, 2, (256,), generator=torch.Generator().manual_seed(1)).float()
    steps = (torch.randint(-3, 4, (256,), generator=torch.Generator().manual_seed(2)) * 0.001).float()
    for bias in (None, torch.zeros(256), torch.full((256,), 0.25), steps):
        for score in ("sigmoid", "softmax"):
            for groups, top in ((1, 1), (8, 4)):
                check(cuda_device, x, 8, bias, score, groups, top, "top2")
                check(cuda_device, x.bfloat16(), 32, bias, score, groups, top, "max")
    ids, _ = check(cuda_device, x[:1], 8)
    assert ids[0].tolist() == list(range(8))


def test_large_and_small_logits(cuda_device):
    """Scores at 0 and 1 in FP32: the order of the logits without a bias, ratios of tiny scores with renormalisation."""
    x = torch.stack((torch.linspace(-120, -95, 64), torch.linspace(80, 30, 64), torch.linspace(-300, 300, 64)))
    for renorm in (True, False):
        for score in ("sigmoid", "softmax"):
            ids, w = check(cuda_device, x, 6, None, score, renorm=renorm)
            assert bool(torch.isfinite(w).all())
    check(cuda_device, x[1:], 6, torch.linspace(0, 1e-3, 64), "sigmoid")


def test_absent_experts(cuda_device):
    x = randn(5, 64, seed=9)
    x[0, 5:] = float("-inf")
    x[1, ::2] = float("nan")
    x[2] = float("nan")
    bias = randn(64, std=0.1)
    bias[10:30] = float("-inf")
    bias[40] = float("nan")
    for b in (None, bias):
        for groups, top in ((1, 1), (4, 2)):
            for score in ("sigmoid", "softmax"):
                check(cuda_device, x, 8, b, score, groups, top, "max")
                assert moe.device_error(cuda_device) == 0x4
    check(cuda_device, x[3:], 8, bias)
    every = torch.full((64,), float("-inf"))
    ids, w = moe.router_grouped_topk(x.to(cuda_device), 2, every.to(cuda_device))
    assert bool((ids == -1).all()) and bool((w == 0).all())
    assert moe.device_error(cuda_device) == 0x4


def test_outputs_stay_in_bounds(cuda_device):
    T, E, k = 9, 200, 6
    ids = torch.full((T * k + 64,), -12345, dtype=torch.int32, device=cuda_device)
    w = torch.full((T * k + 64,), -7.0, device=cuda_device)
    x = randn(T, E, seed=4)
    moe.router_grouped_topk(x.to(cuda_device), k, None, "softmax", topk_ids=ids[32:32 + T * k].view(T, k),
                            topk_w=w[32:32 + T * k].view(T, k))
    rid, _ = refs.router(x, k, None, "softmax", 1, 1, "max", True, 1.0)
    assert np.array_equal(ids[32:32 + T * k].view(T, k).cpu().numpy(), rid)
    for t, v in ((ids, -12345), (w, -7.0)):
        assert bool((t[:32] == v).all()) and bool((t[32 + T * k:] == v).all())


def test_captured_and_on_another_stream(cuda_device):
    x, bias = randn(64, 256, seed=5).to(cuda_device), randn(256, std=0.1).to(cuda_device)
    call = lambda: moe.router_grouped_topk(x, 8, bias, "sigmoid", 8, 4, scale=2.5)  # noqa: E731
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    torch.cuda.synchronize()
    for o in (other, got):
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


MANY = 5003   # rows for all SMs' warps: eight lanes a row where the shape allows


@pytest.mark.parametrize("E,k,groups,top", [(32, 8, 1, 1), (32, 2, 8, 3), (64, 6, 4, 2), (96, 5, 1, 1), (128, 8, 8, 4), (160, 7, 4, 1),
                                            (224, 1, 2, 1), (256, 8, 8, 4), (256, 8, 1, 1), (256, 3, 16, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_many_rows(cuda_device, E, k, groups, top, dtype):
    x = randn(MANY, E, seed=E + k, dtype=dtype)
    for score, gs, bias, renorm in (("sigmoid", "top2", True, True), ("softmax", "max", True, False), ("sigmoid", "top2", False, False),
                                    ("softmax", "top2", False, True), ("sigmoid", "max", False, True)):
        b = randn(E, seed=E, std=0.1 if score == "sigmoid" else 0.3 / E) if bias else None
        check(cuda_device, x, k, b, score, groups, top, gs, renorm, 2.5, f"{score} {gs} bias={bias}")


def test_many_rows_with_ties_absences_and_near_keys(cuda_device):
    g = torch.Generator().manual_seed(11)
    E = 256
    steps = (torch.randint(-3, 4, (E,), generator=g) * 0.001).float()
    ties = torch.randint(0, 5, (MANY, E), generator=g).float()
    few = randn(MANY, E, seed=12)
    few[::7, 3:] = float("-inf")
    few[1::7, ::2] = float("nan")
    hole = randn(E, seed=13, std=0.1)
    hole[64:200] = float("-inf")
    p = torch.sigmoid(few[0:1].nan_to_num(0, neginf=0)).double()
    near = few[0:1].nan_to_num(0, neginf=0) + 1e-6 * randn(MANY, E, seed=14)
    nb = (0.75 - p[0]).float()
    for groups, top in ((1, 1), (8, 4)):
        check(cuda_device, ties, 8, None, "sigmoid", groups, top, what="ties")
        check(cuda_device, ties, 8, steps, "softmax", groups, top, "max", what="ties and steps")
        check(cuda_device, ties.bfloat16(), 4, torch.zeros(E), "sigmoid", groups, top, what="ties, zeros")
        check(cuda_device, near, 8, nb, "sigmoid", groups, top, what="near")
        check(cuda_device, randn(MANY, E, seed=15), 8, hole, "sigmoid", groups, top, "max", what="hole")
        assert moe.device_error(cuda_device) == 0
        check(cuda_device, few, 8, None, "softmax", groups, top, "max", what="few")
        assert moe.device_error(cuda_device) == 0x4


def test_many_rows_with_a_row_stride(cuda_device):
    base = randn(MANY, 300, seed=16)
    for at, E in ((0, 256), (4, 128), (1, 64)):
        x = base[:, at:at + E]
        b = randn(E, seed=E, std=0.1)
        ids, w = moe.router_grouped_topk(base.to(cuda_device)[:, at:at + E], 6, b.to(cuda_device), "sigmoid", 4, 2)
        rid, rw = refs.router(x, 6, b, "sigmoid", 4, 2, "top2", True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), rid)
        np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=2.0 ** -20)
