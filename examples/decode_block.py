"""One decoder block, token by token, on this library's operators.

The block around the expert layer: norm, 4-bit projections, head norms, rotary
positions with the cache append, paged attention, output projection, residual
and norm, router, expert layer.  A decode step is one CUDA graph: positions,
page slots and lengths live on the device and move on inside it.  Three things
are torch calls: the router's small projection, the slots and lengths of the new
tokens, and the conversion of the 32-bit stream for the first norm.

    python examples/decode_block.py [--batch 8] [--context 4096] [--steps 64]

Random weights of a Qwen3-style block (E=128, top-8, d=2048, I=768; 32 query
and 4 key-value heads of 128).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_decode_gb300 as moe  # noqa: E402
from mixture_experts_decode_gb300 import inputs  # noqa: E402

BF = torch.bfloat16


def pack4(w: torch.Tensor, group: int) -> moe.W4:
    """Round-to-nearest 4-bit weights with a zero point per group, from float [N, K]."""
    N, K = w.shape
    g = w.float().view(N, K // group, group)
    lo, hi = g.amin(-1), g.amax(-1)
    scale = ((hi - lo) / 15).clamp_min(1e-8).to(BF)
    zero = torch.round(-lo / scale.float()).clamp(0, 15)
    code = torch.round(g / scale.float()[..., None] + zero[..., None]).clamp(0, 15).to(torch.uint8).view(N, K)
    return moe.W4((code[:, 0::2] | code[:, 1::2] << 4).contiguous(), scale.contiguous(), zero.to(torch.uint8).contiguous())


def first_slots(table: torch.Tensor, page: int, pages: int) -> torch.Tensor:
    """Slot of the first row of each page of a sequence, and behind them one past the cache: a token of a sequence
    whose pages are full is not written, and the library reports it (device_error) as it does the length."""
    past = torch.full_like(table[:, :1], pages)
    return torch.cat((table, past), 1).long() * page


def cache_slots(first: torch.Tensor, positions: torch.Tensor, page: int) -> torch.Tensor:
    """Slot of each sequence's next token."""
    at = (positions // page).clamp(max=first.shape[1] - 1).long()
    return torch.gather(first, 1, at[:, None])[:, 0] + positions % page


class DecodeBlock:
    """Weights of one block and the pages of its cache for up to `batch` sequences of `capacity` tokens."""

    def __init__(self, cfg: inputs.LayerConfig, Hq: int, Hkv: int, D: int, batch: int, capacity: int, page: int = 64,
                 device="cuda", seed: int = 0, group: int = 128):
        self.cfg, self.Hq, self.Hkv, self.D, self.page = cfg, Hq, Hkv, D, page
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s, std=0.02: torch.randn(*s, generator=g, device=device) * std  # noqa: E731
        norm = lambda n: moe.Norm((1 + rnd(n, std=0.1)).to(BF))  # noqa: E731
        self.attn_norm, self.moe_norm = norm(cfg.d), norm(cfg.d)
        self.q_norm, self.k_norm = norm(D), norm(D)
        self.wq, self.wk, self.wv = (pack4(rnd(h * D, cfg.d), group) for h in (Hq, Hkv, Hkv))
        self.wo = pack4(rnd(cfg.d, Hq * D), group)
        self.router = rnd(cfg.E, cfg.d)
        W = inputs.layer_weights(cfg, device)
        self.experts = [moe.MX(W["w_" + n], W["s_" + n]) for n in ("gate", "up", "down")]
        self.freqs = moe.rope_freqs(D, base=1000000.0, device=device)
        most = -(-capacity // page)
        pages = batch * most
        self.k_cache = torch.zeros(pages, page, Hkv, D, dtype=BF, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.table = torch.randperm(pages, generator=g, device=device).view(batch, most).to(torch.int32)
        self.first = first_slots(self.table, page, pages)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.workspace = moe.attention_workspace(Hq, Hkv, D, device)

    def step(self, resid: torch.Tensor) -> torch.Tensor:
        """One new token for every sequence: resid float32 [B, d] in and out (in place)."""
        B = resid.shape[0]
        positions = self.lens.clone()
        slots = cache_slots(self.first, positions, self.page)
        self.lens += 1

        # (the first norm has nothing to add: the residual stream is its input)
        x = moe.norm_residual(resid.to(BF), pre=self.attn_norm)
        q = moe.matvec4(x, self.wq).view(B * self.Hq, self.D)
        k = moe.matvec4(x, self.wk).view(B * self.Hkv, self.D)
        v = moe.matvec4(x, self.wv).view(B, self.Hkv, self.D)
        q = moe.norm_residual(q, pre=self.q_norm).view(B, self.Hq, self.D)
        k = moe.norm_residual(k, pre=self.k_norm).view(B, self.Hkv, self.D)
        q = moe.rope_append(q, k, v, positions, slots, self.freqs, self.k_cache, self.v_cache, q_out=q)
        a = moe.paged_attention(q, self.k_cache, self.v_cache, self.table, self.lens, workspace=self.workspace)
        o = moe.matvec4(a.view(B, -1), self.wo)
        _, x = moe.norm_residual(o, resid, pre=self.moe_norm, resid_out=resid)
        ids, w = moe.router_topk(x.float() @ self.router.T, self.cfg.k)
        y = moe.layer(x, ids, w, *self.experts)
        moe.norm_residual(y, resid, resid_out=resid)
        return resid


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--context", type=int, default=4096, help="tokens in the cache before the first step")
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    block = DecodeBlock(inputs.QWEN3, 32, 4, 128, a.batch, a.context + a.steps + 16)
    block.k_cache.normal_()
    block.v_cache.normal_()
    resid = torch.randn(a.batch, inputs.QWEN3.d, device="cuda")
    block.lens.fill_(a.context)
    for _ in range(3):
        block.step(resid)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(resid)
    block.lens.fill_(a.context)
    graph.replay()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert moe.device_error() == 0 and bool(torch.isfinite(resid).all())
    print(f"{a.batch} sequences of {a.context} tokens: {begin.elapsed_time(end) / a.steps * 1e3:.1f} us a block and step, "
          f"lengths now {block.lens.tolist()[0]}")


if __name__ == "__main__":
    main()
