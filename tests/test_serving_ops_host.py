"""The serving step's entry points on the host (no GPU): refusals before any launch."""
import pytest
import torch

import mixture_experts_decode_gb300 as moe

ARG, SHAPE, LIMIT, WORKSPACE, ALIGN = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_decode_gb300 import build
    build.build()
    return moe.load()


def _router(lib, x=0x10000, stride=64, T=4, E=64, dtype=2, bias=0x20000, k=4, score=1, groups=8, top=4, gs=1, renorm=1,
            ids=0x30000, w=0x40000):
    return lib.moe_router_grouped_topk(x, stride, T, E, dtype, bias, k, score, groups, top, gs, renorm, 1.0, ids, w, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), ARG), (dict(E=0), ARG), (dict(k=0), ARG), (dict(groups=0), ARG), (dict(top=0), ARG), (dict(dtype=3), ARG),
    (dict(score=2), ARG), (dict(gs=2), ARG), (dict(renorm=2), ARG), (dict(groups=7), SHAPE), (dict(top=9), SHAPE),
    (dict(k=9, top=1), SHAPE), (dict(E=8), SHAPE), (dict(E=2048), LIMIT), (dict(E=1024, k=33), LIMIT),
    (dict(E=1024, groups=64), LIMIT), (dict(x=None), ARG), (dict(ids=None), ARG), (dict(w=None), ARG),
    (dict(x=0x10002), ALIGN), (dict(dtype=0, x=0x10001), ALIGN), (dict(bias=0x20002), ALIGN), (dict(ids=0x30001), ALIGN),
    (dict(w=0x40002), ALIGN),
])
def test_router_refusals(lib, kw, rc):
    assert _router(lib, **kw) == rc


def test_router_of_no_tokens_launches_nothing(lib):
    assert _router(lib, T=0, x=None, ids=None, w=None) == 0


def _plan(lib, past=0x10000, new=0x11000, B=4, table=0x20000, most=8, free=0x30000, cap=16, n=0x31000, page=16, shared=None,
          ns=0, T=8, pos=0x40000, slots=0x41000, seq=0x42000, starts=0x43000, lens=0x44000, left=0x45000):
    return lib.moe_plan_pages(past, new, B, table, most, most, free, cap, n, page, shared, ns, None, T, pos, slots, seq, starts,
                              lens, left, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(most=-1), ARG), (dict(cap=-1), ARG), (dict(page=0), ARG), (dict(ns=-1), ARG),
    (dict(B=4097), LIMIT), (dict(past=None), ARG), (dict(new=None), ARG), (dict(lens=None), ARG), (dict(table=None), ARG),
    (dict(n=None), ARG), (dict(left=None), ARG), (dict(starts=None), ARG), (dict(free=None), ARG), (dict(ns=2), ARG),
    (dict(pos=None), ARG), (dict(slots=None), ARG), (dict(seq=None), ARG), (dict(past=0x10002), ALIGN),
    (dict(slots=0x41004), ALIGN), (dict(left=0x45001), ALIGN), (dict(table=0x20002), ALIGN),
])
def test_plan_refusals(lib, kw, rc):
    assert _plan(lib, **kw) == rc


def _release(lib, table=0x20000, most=8, lens=0x10000, B=4, ended=0x11001, free=0x30000, cap=16, n=0x31000, page=16, ns=0,
             out=0x44000, left=0x45000):
    return lib.moe_release_pages(table, most, most, lens, B, ended, free, cap, n, page, ns, None, out, left, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), ARG), (dict(most=-1), ARG), (dict(cap=-1), ARG), (dict(page=0), ARG), (dict(ns=-1), ARG), (dict(B=4097), LIMIT),
    (dict(lens=None), ARG), (dict(ended=None), ARG), (dict(out=None), ARG), (dict(table=None), ARG), (dict(n=None), ARG),
    (dict(left=None), ARG), (dict(free=None), ARG), (dict(lens=0x10002), ALIGN), (dict(out=0x44002), ALIGN),
])
def test_release_refusals(lib, kw, rc):
    assert _release(lib, **kw) == rc


def test_binding_refuses_mismatched_tensors(lib):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(3, 64)
    with pytest.raises(TypeError):
        moe.router_grouped_topk(x.double(), 4)
    with pytest.raises(ValueError):
        moe.router_grouped_topk(x, 4, torch.zeros(32))
    with pytest.raises(TypeError):
        moe.router_grouped_topk(x, 4, torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        moe.router_grouped_topk(x.T, 2)
    with pytest.raises(KeyError):
        moe.router_grouped_topk(x, 4, score="tanh")
    with pytest.raises(ValueError):
        moe.router_grouped_topk(x, -1)
    with pytest.raises(ValueError):
        moe.router_grouped_topk(x, 4)           # not on a GPU
    with pytest.raises(TypeError):
        moe.plan_pages(i(2).long(), i(2), i(2, 4), i(8), i(1), 16, 2)
    with pytest.raises(ValueError):
        moe.plan_pages(i(2), i(3), i(2, 4), i(8), i(1), 16, 2)
    with pytest.raises(ValueError):
        moe.plan_pages(i(2), i(2), i(3, 4), i(8), i(1), 16, 2)
    with pytest.raises(ValueError):
        moe.plan_pages(i(2), i(2), i(2, 4), i(8), i(2), 16, 2)
    with pytest.raises(ValueError):
        moe.plan_pages(i(2), i(2), i(2, 4), i(8), i(1), 16, -2)
    with pytest.raises(TypeError):
        moe.plan_pages(i(2), i(2), i(2, 4), i(8), i(1), 16, 2, shares=i(2))
    with pytest.raises(ValueError):
        moe.plan_pages(i(2), i(2), i(2, 4), i(8), i(1), 16, 2)   # not on a GPU
    with pytest.raises(ValueError):
        moe.release_pages(i(2, 4), i(2), torch.zeros(3, dtype=torch.bool), i(8), i(1), 16)
    with pytest.raises(TypeError):
        moe.release_pages(i(2, 4), i(2), i(2), i(8), i(1), 16)
