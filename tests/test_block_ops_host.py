"""The decode block's entry points on the host (no GPU): refusals before any launch, and moe_rope_freqs."""
import ctypes
import math

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


def _attn(lib, q=0x20000, qs=256, qh=64, B=2, Hq=4, Hkv=2, D=64, dtype=0, k=None, v=None, cdt=0, pages=8, page=16,
          table=0x30000, most=4, lens=0x40000, window=0, sinks=0, ws=0x50000, wsb=1 << 30, out=0x60000, lse=None):
    return lib.moe_paged_attention(q, qs, qh, B, Hq, Hkv, D, dtype, k or _kv(), v or _kv(), cdt, pages, page, table, most,
                                   most, lens, 0.1, window, sinks, ws, wsb, out, lse, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), ARG), (dict(Hq=0), ARG), (dict(Hkv=0), ARG), (dict(D=0), ARG), (dict(page=0), ARG), (dict(pages=-1), ARG),
    (dict(most=-1), ARG), (dict(window=-1), ARG), (dict(sinks=-1), ARG), (dict(dtype=2), ARG), (dict(dtype=3), ARG),
    (dict(cdt=1), ARG), (dict(cdt=7), ARG), (dict(dtype=1, cdt=0), ARG), (dict(Hq=5), SHAPE), (dict(D=72), SHAPE),
    (dict(D=272), LIMIT), (dict(B=1025), LIMIT), (dict(q=None), ARG), (dict(lens=None), ARG), (dict(out=None), ARG),
    (dict(table=None), ARG), (dict(k=_kv(None)), ARG), (dict(ws=None), WORKSPACE), (dict(wsb=1000), WORKSPACE),
    (dict(ws=0x50080), ALIGN), (dict(q=0x20008), ALIGN), (dict(qs=260), ALIGN), (dict(qh=68), ALIGN),
    (dict(k=_kv(0x10008)), ALIGN), (dict(v=_kv(token=260)), ALIGN), (dict(cdt=3, k=_kv(head=72)), ALIGN),
    (dict(out=0x60001), ALIGN), (dict(lse=0x70002), ALIGN), (dict(lens=0x40002), ALIGN),
])
def test_attention_refusals(lib, kw, rc):
    assert _attn(lib, **kw) == rc


def test_attention_of_no_sequences_launches_nothing(lib):
    assert _attn(lib, B=0) == 0


def test_attention_workspace_bytes(lib):
    n = ctypes.c_size_t()
    assert lib.moe_paged_attention_workspace_bytes(32, 4, 128, ctypes.byref(n)) == 0
    # a counter page, and two pieces of 8 heads x (128 + 2) floats for each of 480 blocks
    assert n.value == -(-(4096 + 2 * 480 * 8 * 130 * 4) // 256) * 256
    assert lib.moe_paged_attention_workspace_bytes(32, 4, 128, None) == ARG
    assert lib.moe_paged_attention_workspace_bytes(33, 4, 128, ctypes.byref(n)) == SHAPE
    assert lib.moe_paged_attention_workspace_bytes(32, 4, 512, ctypes.byref(n)) == LIMIT


def _rope(lib, q=0x20000, k=0x21000, v=0x22000, T=2, Hq=4, Hkv=2, D=64, dtype=0, pos=0x30000, slots=0x31000, freqs=0x32000,
          rot=64, inter=0, kc=None, vc=None, cdt=0, pages=8, page=16, out=0x60000):
    return lib.moe_rope_append(q, 256, 64, k, 128, 64, v, 128, 64, T, Hq, Hkv, D, dtype, pos, slots, freqs, rot, inter, 1.0,
                               kc or _kv(), vc or _kv(), cdt, pages, page, out, 256, 64, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), ARG), (dict(Hq=0), ARG), (dict(D=0), ARG), (dict(rot=-2), ARG), (dict(page=0), ARG), (dict(dtype=2), ARG),
    (dict(cdt=1), ARG), (dict(inter=2), ARG), (dict(rot=33), SHAPE), (dict(rot=66), SHAPE), (dict(D=514), LIMIT),
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(pos=None), ARG), (dict(slots=None), ARG),
    (dict(freqs=None), ARG), (dict(out=None), ARG), (dict(kc=_kv(None)), ARG), (dict(q=0x20001), ALIGN),
    (dict(kc=_kv(0x10001)), ALIGN), (dict(slots=0x31004), ALIGN), (dict(freqs=0x32004), ALIGN), (dict(pos=0x30002), ALIGN),
])
def test_rope_refusals(lib, kw, rc):
    assert _rope(lib, **kw) == rc


def test_rope_of_no_tokens_launches_nothing(lib):
    assert _rope(lib, T=0) == 0


def _norm(lib, y=0x20000, T=2, d=64, dtype=0, r=0x30000, rdt=0, post=None, gate=None, gcol=0, act=0, pre=None, ro=0x40000,
          out=0x50000):
    ref = lambda n: None if n is None else ctypes.byref(n)  # noqa: E731
    return lib.moe_norm_residual(y, 64, T, d, dtype, r, 64, rdt, ref(post), gate, 0, gcol, act, 1.0, ref(pre), ro, out, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), ARG), (dict(d=0), ARG), (dict(dtype=2), ARG), (dict(rdt=1), ARG), (dict(act=2), ARG),
    (dict(gate=0x70000, gcol=2), ARG), (dict(pre=_lib.NormView(None, None, 1e-6, 2)), ARG),
    (dict(post=_lib.NormView(None, None, 1e-6, -1)), ARG), (dict(d=32769), LIMIT), (dict(y=None), ARG),
    (dict(ro=None, out=None), ARG), (dict(y=0x20001), ALIGN), (dict(rdt=2, r=0x30002), ALIGN), (dict(gate=0x70001), ALIGN),
    (dict(rdt=2, ro=0x40002), ALIGN), (dict(pre=_lib.NormView(0x80001, None, 1e-6, 0)), ALIGN),
])
def test_norm_refusals(lib, kw, rc):
    assert _norm(lib, **kw) == rc


def _mv(lib, x=0x20000, xs=256, T=2, K=256, dtype=0, codes=0x30000, scales=0x40000, N=64, group=64, y=0x50000):
    return lib.moe_matvec4(x, xs, T, K, dtype, codes, scales, None, N, group, y, N, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), ARG), (dict(N=-1), ARG), (dict(K=-32), ARG), (dict(dtype=2), ARG), (dict(group=16), SHAPE), (dict(K=0), SHAPE),
    (dict(K=96), SHAPE), (dict(T=257), LIMIT), (dict(x=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG),
    (dict(y=None), ARG), (dict(x=0x20008), ALIGN), (dict(xs=260), ALIGN), (dict(codes=0x30008), ALIGN),
    (dict(scales=0x40001), ALIGN), (dict(y=0x50001), ALIGN),
])
def test_matvec_refusals(lib, kw, rc):
    assert _mv(lib, **kw) == rc


def test_matvec_of_nothing_launches_nothing(lib):
    assert _mv(lib, T=0) == 0 and _mv(lib, N=0) == 0


def test_rope_freqs_values(lib):
    f = moe.rope_freqs(8, base=10000.0)
    # 10000^(-2i/8), by hand
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.allclose(moe.rope_freqs(8, scaling="linear", factor=4.0), f / 4, rtol=1e-14)
    # base 10000 * 2^(8/6): the lowest frequency is divided by 2, the highest kept
    n = moe.rope_freqs(8, scaling="ntk", factor=2.0)
    assert n[0] == 1.0 and math.isclose(n[3].item(), f[3].item() / 2, rel_tol=1e-13)
    # 4096 tokens hold 652, 65, 6.5 and 0.65 turns: kept, kept, on the ramp, divided
    p = moe.rope_freqs(8, scaling="by_parts", factor=8.0, original_length=4096)
    g = (4096 * 0.01 / (2 * math.pi) - 1) / 31
    want = torch.tensor([1.0, 0.1, 0.01 * (g + (1 - g) / 8), 0.001 / 8], dtype=torch.float64)
    assert torch.allclose(p, want, rtol=1e-13)


@pytest.mark.parametrize("kw", [dict(rot=7), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, base=float("nan")),
                                dict(rot=8, scaling="linear", factor=0.0), dict(rot=2, scaling="ntk", factor=2.0),
                                dict(rot=8, scaling="by_parts", factor=2.0, beta_fast=1.0, beta_slow=1.0),
                                dict(rot=8, scaling="by_parts", factor=2.0, original_length=0)])
def test_rope_freqs_refusals(lib, kw):
    with pytest.raises(moe.MoEError):
        moe.rope_freqs(**kw)


def test_binding_refuses_mismatched_tensors(lib):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    tab, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        moe.paged_attention(q.float(), k, k, tab, lens)
    with pytest.raises(TypeError):
        moe.paged_attention(q, k.half(), k.half(), tab, lens)
    with pytest.raises(TypeError):
        moe.paged_attention(q, k, k, tab.long(), lens)
    with pytest.raises(ValueError):
        moe.paged_attention(q, k, k[..., :32], tab, lens)
    with pytest.raises(ValueError):
        moe.paged_attention(q, k, k, tab[:1], lens)
    with pytest.raises(ValueError):
        moe.paged_attention(q, k, k, tab, lens[:1])
    with pytest.raises(ValueError):
        moe.paged_attention(q.transpose(1, 2), k, k, tab, lens)
    with pytest.raises(TypeError):
        moe.rope_append(q, q[:, :2], q[:, :2], lens, lens, torch.ones(32, dtype=torch.float64), k, k)
    with pytest.raises(ValueError):
        moe.rope_append(q, q[:, :1], q[:, :2], lens, lens.long(), torch.ones(32, dtype=torch.float64), k, k)
    y = torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        moe.norm_residual(y, y.bfloat16())
    with pytest.raises(ValueError):
        moe.norm_residual(y, gate=y[:, :3])
    with pytest.raises(ValueError):
        moe.norm_residual(y, pre=moe.Norm(y[0, :32]))
    with pytest.raises(KeyError):
        moe.norm_residual(y, pre=moe.Norm(kind="batch"))
    codes, scales = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.matvec4(y, moe.W4(codes[:, :16].contiguous(), scales))
    with pytest.raises(TypeError):
        moe.matvec4(y, moe.W4(codes, scales.bfloat16()))
    with pytest.raises(ValueError):
        moe.matvec4(y, moe.W4(codes, scales, torch.zeros(8, 1, dtype=torch.uint8)))


def test_attention_needs_a_table_even_without_pages(lib):
    assert _attn(lib, pages=0, table=None) == ARG
    assert _attn(lib, pages=0, k=_kv(None), v=_kv(None), table=None) == ARG
