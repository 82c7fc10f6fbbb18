"""One decoder block, token by token, on this library's operators.

The block around the expert layer: norm, 4-bit projections, head norms, rotary
positions with the cache append, paged attention, output projection, residual
and norm, router, expert layer.  A decode step is one CUDA graph: positions,
page slots and lengths live on the device and move on inside it.  Three things
are torch calls: the router's small projection, the slots and lengths of the new
tokens, and the conversion of the 32-bit stream for the first norm.

With --shared N the sequences begin with the same N tokens and live in a pool of
pages: SharedBlock plans pages, slots and lengths on the device, reads the shared
prefix once for all sequences, and routes with a balancing bias within groups.

    python examples/decode_block.py [--batch 8] [--context 4096] [--steps 64] [--shared 0]

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

    def place(self, B: int):
        """Positions and slots of the new tokens; the lengths move on."""
        positions = self.lens.clone()
        slots = cache_slots(self.first, positions, self.page)
        self.lens += 1
        return positions, slots

    def attend(self, q: torch.Tensor) -> torch.Tensor:
        return moe.paged_attention(q, self.k_cache, self.v_cache, self.table, self.lens, workspace=self.workspace)

    def route(self, logits: torch.Tensor):
        return moe.router_topk(logits, self.cfg.k)

    def step(self, resid: torch.Tensor) -> torch.Tensor:
        """One new token for every sequence: resid float32 [B, d] in and out (in place)."""
        B = resid.shape[0]
        positions, slots = self.place(B)

        # (the first norm has nothing to add: the residual stream is its input)
        x = moe.norm_residual(resid.to(BF), pre=self.attn_norm)
        q = moe.matvec4(x, self.wq).view(B * self.Hq, self.D)
        k = moe.matvec4(x, self.wk).view(B * self.Hkv, self.D)
        v = moe.matvec4(x, self.wv).view(B, self.Hkv, self.D)
        q = moe.norm_residual(q, pre=self.q_norm).view(B, self.Hq, self.D)
        k = moe.norm_residual(k, pre=self.k_norm).view(B, self.Hkv, self.D)
        q = moe.rope_append(q, k, v, positions, slots, self.freqs, self.k_cache, self.v_cache, q_out=q)
        a = self.attend(q)
        o = moe.matvec4(a.view(B, -1), self.wo)
        _, x = moe.norm_residual(o, resid, pre=self.moe_norm, resid_out=resid)
        ids, w = self.route(x.float() @ self.router.T)
        y = moe.layer(x, ids, w, *self.experts)
        moe.norm_residual(y, resid, resid_out=resid)
        return resid


class SharedBlock(DecodeBlock):
    """The block for sequences that begin with the same `shared` tokens (whole pages), over a pool of pages.

    begin() starts a sequence behind the prefix, or without it; end() marks those whose pages go back to the pool at
    the next step.  Both take effect there, the ends first, so that a slot may end and begin again between two steps.
    The prefix's keys and values are the pages self.shared of the caches."""

    def __init__(self, cfg: inputs.LayerConfig, Hq: int, Hkv: int, D: int, batch: int, capacity: int, shared: int,
                 page: int = 64, device="cuda", seed: int = 0, group: int = 128, groups: int = 1, top_groups: int = 1):
        super().__init__(cfg, Hq, Hkv, D, batch, capacity, page, device, seed, group)
        assert shared % page == 0 and shared <= capacity
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
        n = shared // page
        order = self.table.flatten()
        self.shared, self.shared_len, self.batch = order[:n].contiguous(), shared, batch
        self.free, self.n_free = torch.cat((order[n:], order[:n])), i32([order.numel() - n])
        self.table = torch.full_like(self.table, -1)
        self.new = torch.zeros(batch, dtype=torch.int32, device=device)   # a token a step of those that run
        self.shares = torch.ones(batch, dtype=torch.bool, device=device)
        self.ended = torch.zeros(batch, dtype=torch.bool, device=device)
        # what begins at the next step: its length, -1 for none
        self.next_lens = torch.full((batch,), -1, dtype=torch.int32, device=device)
        self.next_shares = torch.ones(batch, dtype=torch.bool, device=device)
        self.runs = [False] * batch
        self.workspace = moe.shared_prefix_workspace(batch, Hq, Hkv, D, device)
        self.groups, self.top_groups = groups, top_groups
        self.bias = torch.zeros(cfg.E, device=device)

    def begin(self, b: int, shares: bool = True):
        if self.runs[b]:
            raise ValueError(f"sequence {b} runs: end it first")
        self.runs[b] = True
        self.next_shares[b], self.new[b] = shares, 1
        self.next_lens[b] = self.shared_len if shares else 0

    def end(self, b: int):
        self.runs[b] = False
        self.ended[b] = True
        self.next_lens[b], self.new[b] = -1, 0

    def place(self, B: int):
        moe.release_pages(self.table, self.lens, self.ended, self.free, self.n_free, self.page, shared=self.shared.numel(),
                          shares=self.shares, seq_lens_out=self.lens, n_free_out=self.n_free)
        self.ended.zero_()
        begins = self.next_lens >= 0
        self.lens.copy_(torch.where(begins, self.next_lens, self.lens))
        self.shares.copy_(torch.where(begins, self.next_shares, self.shares))
        self.next_lens.fill_(-1)
        # one row a sequence: those that do not run bring no token, and their rows behind the last token are padding
        p = moe.plan_pages(self.lens, self.new, self.table, self.free, self.n_free, self.page, B, shared_pages=self.shared,
                           shares=self.shares, seq_lens=self.lens, n_free_out=self.n_free)
        at = p.starts[:-1].long().clamp(max=B - 1)   # (the block's rows are the sequences', not the plan's tokens)
        runs = p.starts[1:] > p.starts[:-1]
        return torch.where(runs, p.positions[at], 0), torch.where(runs, p.slots[at], -1)

    def attend(self, q: torch.Tensor) -> torch.Tensor:
        return moe.shared_prefix_attention(q, self.k_cache, self.v_cache, self.shared, self.shared_len, self.table, self.lens,
                                           shares=self.shares, workspace=self.workspace)

    def route(self, logits: torch.Tensor):
        return moe.router_grouped_topk(logits, self.cfg.k, self.bias, "softmax", self.groups, self.top_groups)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--context", type=int, default=4096, help="tokens in the cache before the first step")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--shared", type=int, default=0, help="tokens of a shared prefix that the sequences begin with")
    a = ap.parse_args()
    if a.shared:
        block = SharedBlock(inputs.QWEN3, 32, 4, 128, a.batch, a.shared + a.steps + 128, a.shared // 64 * 64)
        start = lambda: [block.begin(b) for b in range(a.batch)]  # noqa: E731
        a.context = block.shared_len
    else:
        block = DecodeBlock(inputs.QWEN3, 32, 4, 128, a.batch, a.context + a.steps + 16)
        start = lambda: block.lens.fill_(a.context)  # noqa: E731
    block.k_cache.normal_()
    block.v_cache.normal_()
    resid = torch.randn(a.batch, inputs.QWEN3.d, device="cuda")
    start()
    for _ in range(3):
        block.step(resid)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(resid)
    if not a.shared:
        start()
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
