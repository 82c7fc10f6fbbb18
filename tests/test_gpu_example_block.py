"""The example's decoder block against the same block in 64 bits, step by step and as a graph.

Ten BF16 roundings lie between the residual stream before and after a step
(norm, projections, head norm, rotary, attention, output projection, norm, h
and y of the expert layer, the stream itself as BF16 into the norm), each at
most 2^-9 of its tensor's size in the 2-norm sense (half a step of 2^-8 at
worst); the update of the stream may be off by their sum, 10 * 2^-8 of its own
size, and the 64-bit block starts every step from the GPU's stream and cache,
so nothing adds up over steps.  The router's choice is taken from the GPU's
own norm output, which is compared by itself."""
import os
import sys

import pytest
import torch

import mixture_experts_decode_gb300 as moe
from mixture_experts_decode_gb300 import inputs

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_block  # noqa: E402

pytestmark = pytest.mark.gpu


def rms(x, n):
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + n.eps) * n.w.double()


def dense(w: moe.W4):
    N, half = w.codes.shape
    c = torch.stack((w.codes & 15, w.codes >> 4), -1).view(N, -1, 2 * half // w.scales.shape[1]).double()
    return ((c - w.zeros.double()[..., None]) * w.scales.double()[..., None]).view(N, -1)


def mx(m: moe.MX):
    scale = torch.exp2(m.s.double() - 127)
    return m.w.view(torch.float8_e4m3fn).double() * scale.repeat_interleave(32, -1)


def rope(x, pos, freqs):
    a = pos.double()[:, None, None] * freqs
    u, v = x.chunk(2, -1)
    return torch.cat((u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()), -1)


def reference(b, resid, lens):
    """The update of the residual stream by one step, from the block's present cache."""
    B, Hq, Hkv, D = resid.shape[0], b.Hq, b.Hkv, b.D
    x = rms(resid, b.attn_norm)
    q = rope(rms((x @ dense(b.wq).T).view(B, Hq, D), b.q_norm), lens, b.freqs)
    k = rope(rms((x @ dense(b.wk).T).view(B, Hkv, D), b.k_norm), lens, b.freqs)
    v = (x @ dense(b.wv).T).view(B, Hkv, D)
    out = torch.empty(B, Hq, D, dtype=torch.float64, device=resid.device)
    for i in range(B):
        n = int(lens[i])
        rows = b.table[i].long()
        kk = torch.cat((b.k_cache[rows].flatten(0, 1)[:n].double(), k[i:i + 1]))
        vv = torch.cat((b.v_cache[rows].flatten(0, 1)[:n].double(), v[i:i + 1]))
        for h in range(Hq):
            p = torch.softmax(kk[:, h // (Hq // Hkv)] @ q[i, h] * D ** -0.5, 0)
            out[i, h] = p @ vv[:, h // (Hq // Hkv)]
    o = out.view(B, -1) @ dense(b.wo).T
    return o, rms(resid.double() + o, b.moe_norm)


def test_block_steps_and_graph(cuda_device):
    cfg = inputs.TINY
    b = decode_block.DecodeBlock(cfg, 4, 2, 64, batch=3, capacity=90, page=16, device=cuda_device, group=64)
    b.k_cache.normal_()
    b.v_cache.normal_()
    b.lens.copy_(torch.tensor([0, 15, 70], dtype=torch.int32))
    resid = torch.randn(3, cfg.d, device=cuda_device)
    gate, up, down = (mx(m) for m in b.experts)
    seen = []
    layer = moe.layer
    graph = None
    try:
        decode_block.moe.layer = lambda x, ids, w, *e, **kw: (seen.append((x, ids, w)), layer(x, ids, w, *e, **kw))[1]
        for step in range(6):
            before, lens = resid.clone(), b.lens.clone()
            o, x_ref = reference(b, before, lens)
            if step < 3:
                b.step(resid)
            else:
                if graph is None:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):     # (records, does not run)
                        b.step(resid)
                graph.replay()
            torch.cuda.synchronize()
            x, ids, w = seen[-1]
            assert torch.equal(b.lens, lens + 1)
            err = (x.double() - x_ref).norm() / x_ref.norm()
            assert err <= 10 * 2.0 ** -8, f"step {step}: the expert layer's input is {err:.3g} off"
            xd = x.double()
            y = torch.zeros_like(xd)
            for i in range(3):
                for e, we in zip(ids[i].tolist(), w[i].double().tolist()):
                    g, u = gate[e] @ xd[i], up[e] @ xd[i]
                    y[i] += we * (down[e] @ (g * torch.sigmoid(g) * u))
            want = o + y
            err = (resid.double() - before.double() - want).norm() / want.norm()
            assert err <= 10 * 2.0 ** -8, f"step {step}: the update is {err:.3g} off"
    finally:
        decode_block.moe.layer = layer
    assert moe.device_error(cuda_device) == 0
