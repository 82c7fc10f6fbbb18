"""The serving step's entry points on the host (no GPU): refusals before any launch."""
import pytest
import torch

import mixture_experts_decode_gb300 as moe
from mixture_experts_decode_gb300 import _lib

ARG, SHAPE, LIMIT, WORKSPACE, ALIGN = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_decode_gb300 import build
    build.build()
    return moe.load()


def _kv(addr=0x10000, page=4096, token=256, head=64, scale=1.0):
    return _lib.CacheView(addr, page, token, head, scale)


def _prefix(lib, q=0x20000, qs=256, qh=64, B=2, Hq=4, Hkv=2, D=64, dtype=0, k=None, v=None, cdt=0, pages=8, page=16,
            shared=0x25000, ns=3, n=40, shares=None, table=0x30000, most=4, lens=0x40000, ws=0x50000, wsb=1 << 30, out=0x60000,
            lse=None):
    return lib.moe_shared_prefix_attention(q, qs, qh, B, Hq, Hkv, D, dtype, k or _kv(), v or _kv(), cdt, pages, page, shared, ns,
                                           n, shares, table, most, most, lens, 0.1, ws, wsb, out, lse, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), ARG), (dict(Hq=0), ARG), (dict(Hkv=0), ARG), (dict(D=0), ARG), (dict(page=0), ARG), (dict(pages=-1), ARG),
    (dict(most=-1), ARG), (dict(ns=-1), ARG), (dict(n=-1), ARG), (dict(dtype=2), ARG), (dict(cdt=1), ARG), (dict(cdt=7), ARG),
    (dict(Hq=5), SHAPE), (dict(D=72), SHAPE), (dict(D=272), LIMIT), (dict(B=1025), LIMIT), (dict(n=49), SHAPE),
    (dict(n=65, ns=9), SHAPE), (dict(n=2 ** 31 - 1, page=2 ** 30, ns=4, most=4), LIMIT), (dict(shared=None), ARG), (dict(shared=0x25002), ALIGN), (dict(q=None), ARG), (dict(lens=None), ARG),
    (dict(out=None), ARG), (dict(table=None), ARG), (dict(k=_kv(None)), ARG), (dict(ws=None), WORKSPACE),
    (dict(wsb=1000), WORKSPACE), (dict(ws=0x50080), ALIGN), (dict(q=0x20008), ALIGN), (dict(qs=260), ALIGN),
    (dict(v=_kv(token=260)), ALIGN), (dict(cdt=3, k=_kv(head=72)), ALIGN), (dict(out=0x60001), ALIGN), (dict(lse=0x70002), ALIGN),
])
def test_prefix_refusals(lib, kw, rc):
    assert _prefix(lib, **kw) == rc


def test_prefix_of_no_sequences_launches_nothing(lib):
    assert _prefix(lib, B=0) == 0


def test_prefix_workspace(lib):
    own = moe.attention_workspace_bytes(32, 4, 128)
    assert moe.shared_prefix_workspace_bytes(0, 32, 4, 128) == own
    # 8 sequences: 64 rows a key-value head, 4 blocks a run of keys, so 40 runs of at most 160 blocks, two pieces each, and the
    # own part, 128 + 2 floats a row
    assert moe.shared_prefix_workspace_bytes(8, 32, 4, 128) >= own + 8 * 32 * (1 + 2 * 40) * 130 * 4
    # more sequences never need less for the same runs, and any batch's is enough for a smaller one
    sizes = [moe.shared_prefix_workspace_bytes(b, 32, 4, 128) for b in (1, 8, 16, 31, 32, 33, 64, 65, 100, 1024)]
    assert sizes == sorted(sizes)
    with pytest.raises(moe.MoEError):
        moe.shared_prefix_workspace_bytes(-1, 32, 4, 128)
    with pytest.raises(moe.MoEError):
        moe.shared_prefix_workspace_bytes(1025, 32, 4, 128)


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
    q, kc = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        moe.shared_prefix_attention(q, kc.half(), kc.half(), i(1), 16, i(2, 4), i(2))
    with pytest.raises(ValueError):
        moe.shared_prefix_attention(q, kc, kc, i(1), 16, i(3, 4), i(2))
    with pytest.raises(ValueError):
        moe.shared_prefix_attention(q, kc, kc, i(1), 16, i(2, 4), i(3))
    with pytest.raises(TypeError):
        moe.shared_prefix_attention(q, kc, kc, i(1).long(), 16, i(2, 4), i(2))
    with pytest.raises(TypeError):
        moe.shared_prefix_attention(q, kc, kc, i(1), 16, i(2, 4), i(2), shares=i(2))
    with pytest.raises(ValueError):
        moe.shared_prefix_attention(q, kc, kc, i(1), 16, i(2, 4), i(2))     # not on a GPU
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
