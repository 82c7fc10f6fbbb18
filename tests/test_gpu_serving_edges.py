"""Edges of the serving step's operators: weights that cancel or lie far below the largest, NaN queries, groups whose keys
cancel, rows on the border of nothing, state updated in place call after call, slots that change hands between two steps."""
import math
import os
import sys

import pytest
import torch

import mixture_experts_decode_gb300 as moe
from mixture_experts_decode_gb300 import inputs
import _block_refs as refs
import _serving_refs as srefs
from test_gpu_router_grouped import MANY, check as check_router, randn
from test_gpu_shared_prefix import BF, E4, HF, call, check, enough, make

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0


def two_kinds(c, every, k_one, k_other, v_one, v_other):
    """Every `every`-th key of the prefix is of one kind, the rest of the other: dim 0 of the keys, all dims of the values."""
    page = c["k"].shape[1]
    for t, one, other in ((c["k"], k_one, k_other), (c["v"], v_one, v_other)):
        x = torch.zeros(c["prefix"], *t.shape[2:], device=t.device)
        dims = slice(0, 1) if t is c["k"] else slice(None)
        x[..., dims] = other
        x[::every, :, dims] = one
        for i, pg in enumerate(c["shared"].tolist()):
            t[pg] = x[i * page:(i + 1) * page].to(t.dtype)
    c["q"].zero_()
    c["ks"] = c["vs"] = 1.0


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (HF, E4), (BF, E4)])
def test_weights_that_cancel(cuda_device, dtype, cache):
    """Half of the keys have value 1 and weight 1, half -1 and a weight a little below it: the output is the difference of
    two sums, so a weight's rounding shows beside it.  Bound: the output's rounding, 2^-17 + 2^-20 of the weights as in
    _block_refs.attention, and half a step of FP32 for each of the keys in a sum."""
    Hkv, D, prefix = 8, 128, 512
    B = enough(Hkv, D, prefix, cache)
    c = make(cuda_device, B, Hkv, Hkv, D, 16, prefix, 0, dtype, cache, seed=41)
    two_kinds(c, 2, 1.0, 0.875, 1.0, -1.0)
    c["q"][..., 0] = 1 + torch.arange(B * Hkv, device=cuda_device).view(B, Hkv) / (B * Hkv)
    out, _ = call(c, scale=2.0 ** -8)
    ro, _, _, _ = refs.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], 2.0 ** -8)
    bound = refs.half_step(dtype) * ro.abs() + 2.0 ** -17 + 2.0 ** -20 + 2 * 512 * 2.0 ** -24
    err = ((out.double() - ro).abs() - bound).max()
    assert err <= 0, f"beyond the bound by {float(err):.3g}"


@pytest.mark.parametrize("dtype,cache,v_tail", [(BF, BF, 6e4), (HF, HF, 6e4), (HF, E4, 448.0), (BF, E4, 448.0)])
@pytest.mark.parametrize("bits", [20, 28, 30])
def test_weights_far_below_the_largest(cuda_device, dtype, cache, v_tail, bits):
    """Keys of value 0 that take nearly all of the weight, 63 of 2^-bits behind each: the output is what is kept of those.
    A weight is held to 2^-38 of the largest (paged_attention's promise; half a step of 2^-24 beside 2^14 times a weight
    that the reference may halve), and FP16 outputs to 2^-25."""
    Hkv, D, prefix = 8, 128, 2048
    B = enough(Hkv, D, prefix, cache)
    c = make(cuda_device, B, Hkv, Hkv, D, 16, prefix, 0, dtype, cache, seed=43)
    two_kinds(c, 64, 8.0, 0.0, 0.0, v_tail)
    c["q"][..., 0] = 1.0
    scale = bits * math.log(2.0) / 8
    out, _ = call(c, scale=scale)
    ro, _, ob, _ = refs.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], scale)
    bound = ob + 2.0 ** -31 * v_tail * 63
    err = ((out.double() - ro).abs() - bound).max()
    assert err <= 0, f"beyond the bound by {float(err):.3g} of {float(ro.abs().max()):.3g}"


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4)])
@pytest.mark.parametrize("prefix", [256, 8192])
def test_queries_that_are_not_finite(cuda_device, prefix, dtype, cache, bad):
    """One value of a head: NaN where paged_attention has it (with and without the prefix), the rest as it was."""
    c = make(cuda_device, 17, 8, 2, 128, 16, prefix, [10 + i for i in range(17)], dtype, cache, seed=47, others=(2,))
    want, wl = call(c)
    for b, h in ((0, 0), (2, 5), (16, 7)):
        c["q"][b, h, 9] = bad
    out, lse = call(c)
    po, pl = moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], k_scale=c["ks"], v_scale=c["vs"], return_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(out), torch.isnan(po)) and torch.equal(torch.isnan(lse), torch.isnan(pl))
    hit = torch.zeros_like(wl, dtype=torch.bool)
    hit[0, 0] = hit[2, 5] = hit[16, 7] = True
    assert bool(torch.isnan(out[hit]).all()) and torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], wl[~hit])


@pytest.mark.parametrize("T", [40, MANY])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_whose_best_keys_cancel(cuda_device, T, score):
    """Two keys near 1000 and -1000 a group: their sum is small, their FP32 roundings are not."""
    E, groups = 64, 8
    bias = torch.full((E,), -2000.0)
    bias[0::8], bias[5::8] = 1000.0, -1000.0
    for top in (1, 3):
        check_router(cuda_device, randn(T, E, seed=51), 6 if top > 1 else 4, bias, score, groups, top, "top2")


@pytest.mark.parametrize("E,groups,top", [(64, 1, 1), (64, 8, 3), (128, 2, 1), (256, 8, 8), (256, 8, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinite_logits_of_many_rows(cuda_device, E, groups, top, score):
    """As for few rows, whatever was in the outputs: with softmax and a bias such a row has no score, so no expert."""
    x, bias = randn(MANY, E, seed=52), randn(E, seed=E, std=0.1)
    x[::9, 3], x[1::50, E - 1] = math.inf, math.inf
    x, k = x.to(cuda_device), 6
    ids = torch.full((MANY, k), -12345, dtype=torch.int32, device=cuda_device)
    w = torch.full((MANY, k), -7.0, device=cuda_device)
    rest = (bias.to(cuda_device), score, groups, top)
    moe.router_grouped_topk(x, k, *rest, topk_ids=ids, topk_w=w)
    few = [moe.router_grouped_topk(part, k, *rest) for part in x.split(1000)]
    torch.cuda.synchronize()
    assert torch.equal(ids, torch.cat([f[0] for f in few]))
    torch.testing.assert_close(w, torch.cat([f[1] for f in few]), rtol=2.0 ** -19, atol=0.0, equal_nan=True)
    none = torch.isinf(x).any(1) & (score == "softmax")
    assert bool((ids[none] == -1).all()) and bool((w[none] == 0).all()) and bool((ids[~none] >= 0).all())
    assert moe.device_error(cuda_device) == (0x4 if score == "softmax" else 0)


def best_us(f):
    for _ in range(3):
        f()
    best = math.inf
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


def test_rows_with_nothing_beyond_the_border_are_not_looked_at_again(cuda_device):
    """Every key of the groups is chosen, or the groups left out are wholly masked: nothing lies close to what is left out."""
    x, bias = randn(65536, 64, seed=53).to(cuda_device), randn(64, std=0.1).to(cuda_device)
    usual = best_us(lambda: moe.router_grouped_topk(x, 7, bias, "sigmoid", 8, 1))
    every = best_us(lambda: moe.router_grouped_topk(x, 8, bias, "sigmoid", 8, 1))
    masked = bias.clone()
    masked[32:] = -math.inf
    none = best_us(lambda: moe.router_grouped_topk(x, 7, masked, "sigmoid", 8, 4))
    print(f"usual {usual:.1f} every {every:.1f} masked {none:.1f} us")
    assert every < 1.6 * usual and none < 1.6 * usual


def test_in_place_plans_and_releases_of_several_blocks_one_after_the_other(cuda_device):
    """Each call reads what the one before has written; prompts and ends of some ten thousand tokens a call, eagerly and
    from a graph."""
    dev, page, most, B = cuda_device, 4, 1000, 48
    g = torch.Generator().manual_seed(57)
    pool = 12000
    free = torch.randperm(pool, generator=g).tolist()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    for graphs in (False, True):
        lens, height, stack = i32([0] * B), i32([pool]), i32(free)
        tab = torch.full((B, most), -1, dtype=torch.int32, device=dev)
        news = [torch.randint(0, 200, (B,), generator=g).tolist() for _ in range(12)]
        ends = [(torch.rand(B, generator=g) < 0.3).tolist() for _ in range(12)]
        d_new, d_end = [i32(n) for n in news], [torch.tensor(e, device=dev) for e in ends]

        def steps():
            got = []
            for n, e in zip(d_new, d_end):
                moe.release_pages(tab, lens, e, stack, height, page, seq_lens_out=lens, n_free_out=height)
                got.append(moe.plan_pages(lens, n, tab, stack, height, page, 10000, seq_lens=lens, n_free_out=height))
                got.append(moe.plan_pages(lens, n, tab, stack, height, page, 10000, seq_lens=lens, n_free_out=height))
            return got

        if graphs:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                plans = steps()
            graph.replay()
        else:
            plans = steps()
        torch.cuda.synchronize()
        h_lens, h_tab, h_stack, h_free, refused = [0] * B, [[-1] * most for _ in range(B)], list(free), pool, False
        for i, (n, e) in enumerate(zip(news, ends)):
            h_stack, h_free, h_lens = srefs.release(h_tab, h_lens, e, h_stack, h_free, page)
            for p in plans[2 * i:2 * i + 2]:
                pos, slots, seqs, starts, h_lens, h_free, h_tab, r = srefs.plan(h_lens, n, h_tab, h_stack, h_free, page, 10000)
                refused |= r
                assert p.starts.tolist() == starts and p.positions.tolist() == pos and p.slots.tolist() == slots, i
        assert lens.tolist() == h_lens and height.tolist() == [h_free] and tab.tolist() == h_tab and stack.tolist() == h_stack
        assert not refused


def test_a_slot_ends_and_begins_again_before_a_step(cuda_device):
    """Between two steps a request ends and another takes its slot (behind the prefix, without it, and given up again):
    the old one's pages go back, the new one begins with its prefix."""
    b = decode_block.SharedBlock(inputs.TINY, 4, 2, 64, batch=3, capacity=112, shared=48, page=16, device=cuda_device, group=64)
    pool = b.k_cache.shape[0] - 3
    resid = torch.randn(3, inputs.TINY.d, device=cuda_device)

    def pages():
        used = []
        for i, n in enumerate(b.lens.tolist()):
            used += b.table[i, 3 if bool(b.shares[i]) else 0:-(-n // 16)].tolist()
        left = b.free[:int(b.n_free)].tolist()
        assert len(set(used + left)) == len(used) + len(left) == pool, "a page lost or held twice"

    for i in range(3):
        b.begin(i, shares=i != 1)
    for _ in range(20):
        b.step(resid)
    assert b.lens.tolist() == [68, 20, 68]
    pages()
    b.end(0)
    b.begin(0, shares=False)
    b.end(1)
    b.begin(1, shares=True)
    b.end(2)
    b.begin(2)
    b.end(2)
    b.step(resid)
    assert b.lens.tolist() == [1, 49, 0]
    pages()
    b.step(resid)
    assert b.lens.tolist() == [2, 50, 0]
    pages()
    with pytest.raises(ValueError, match="runs"):
        b.begin(0)


def test_new_outputs_are_seen_by_dispatch_modes(cuda_device):
    """Outputs that a call makes come from torch's allocating operator, which modes that count or fill memory watch."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.names.append(func.name())
            return func(*args, **(kwargs or {}))

    dev = cuda_device
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    y, x = torch.randn(4, 256, device=dev, dtype=BF), torch.randn(4, 64, device=dev)
    lens, new, tab, stack, height = i32([0, 0]), i32([1, 1]), i32([[-1], [-1]]), i32([0, 1]), i32([2])
    mode = Seen()
    for what, made in ((lambda: moe.norm_residual(y, pre=moe.Norm(None)), 1), (lambda: moe.router_grouped_topk(x, 4), 2),
                       (lambda: moe.plan_pages(lens, new, tab, stack, height, 4, 2), 6)):
        mode.names = []
        with mode:
            what()
        assert sum("aten::empty" in n for n in mode.names) >= made, mode.names


def reads_the_prefix_by_itself(c):
    """Whether a call leaves pieces of the prefix in its workspace, behind what the paged kernel needs."""
    B, Hq, D = c["q"].shape
    Hkv = c["k"].shape[2]
    ws = moe.shared_prefix_workspace(B, Hq, Hkv, D)
    own = moe.attention_workspace_bytes(Hq, Hkv, D)
    ws[own:] = 0xa5
    call(c, ws=ws)
    return not bool((ws[own:] == 0xa5).all())


@pytest.mark.parametrize("B,prefix,Hq,Hkv,D,dtype,cache,by_itself", [
    (4, 16384, 32, 4, 128, BF, E4, True), (4, 16384, 32, 4, 128, HF, E4, True), (3, 65536, 32, 4, 128, BF, E4, False),
    (64, 512, 32, 4, 128, BF, E4, False), (8, 8192, 8, 8, 64, HF, E4, True), (7, 5016, 12, 12, 80, HF, E4, False),
    (8, 2048, 12, 12, 192, HF, E4, False), (32, 512, 32, 4, 128, BF, BF, True), (8, 512, 32, 4, 128, BF, BF, False),
    (16, 512, 8, 8, 64, HF, HF, False)])
def test_the_faster_form_is_taken(cuda_device, B, prefix, Hq, Hkv, D, dtype, cache, by_itself):
    """On either side of the rule, as measured beside it."""
    assert reads_the_prefix_by_itself(make(cuda_device, B, Hq, Hkv, D, 8, prefix, 3, dtype, cache, seed=61)) == by_itself


@pytest.mark.parametrize("D,dtype", [(16, BF), (48, HF), (80, BF), (80, HF), (144, HF), (192, BF), (256, HF)])
def test_codes_of_heads_that_fill_no_block(cuda_device, D, dtype):
    """E4M3 heads of all block numbers by the prefix's kernel."""
    prefix = 24 * 130
    B = math.ceil(70e6 / (2 * prefix * 3 * D)) + 1
    c = make(cuda_device, B, 6, 3, D, 24, prefix, [(i * 7) % 40 for i in range(B)], dtype, E4, seed=D, others=(1,))
    assert reads_the_prefix_by_itself(c)
    check(c, what=f"D={D}")


def test_a_long_prefix_of_codes(cuda_device):
    c = make(cuda_device, 4, 16, 2, 128, 64, 70000, [5, 0, 300, 1], BF, E4, seed=7, q_std=3.0)
    assert reads_the_prefix_by_itself(c)
    check(c, what="long")
