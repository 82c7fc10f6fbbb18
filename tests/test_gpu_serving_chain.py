"""The serving step's operators together, as the example's SharedBlock runs them: pages and slots planned on the device, the
new tokens appended, a shared prefix read once, grouped routing, the expert layer; step by step and as a graph, against 64
bits, with sequences that begin and end on the way.

The update of the residual stream may be off by the ten BF16 roundings between the stream before and after a step, each at
most 2^-8 of its tensor's size in the 2-norm sense (as for the block without a shared prefix)."""
import os
import sys

import pytest
import torch

import mixture_experts_decode_gb300 as moe
from mixture_experts_decode_gb300 import inputs

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_block  # noqa: E402
from test_gpu_example_block import dense, mx, rms, rope  # noqa: E402

pytestmark = pytest.mark.gpu


def reference(b, resid, tokens):
    """(attention's output projection, norm before the experts) in 64 bits; tokens[i]: the (key, value) of each kv head of
    sequence i's tokens so far, appended to here, or None where it does not run."""
    B, Hq, Hkv, D = resid.shape[0], b.Hq, b.Hkv, b.D
    x = rms(resid, b.attn_norm)
    lens = torch.tensor([0 if t is None else len(t[0]) for t in tokens], device=resid.device)
    q = rope(rms((x @ dense(b.wq).T).view(B, Hq, D), b.q_norm), lens, b.freqs)
    k = rope(rms((x @ dense(b.wk).T).view(B, Hkv, D), b.k_norm), lens, b.freqs)
    v = (x @ dense(b.wv).T).view(B, Hkv, D)
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=resid.device)
    for i, t in enumerate(tokens):
        if t is None:
            continue
        kk, vv = torch.cat((t[0], k[i:i + 1])), torch.cat((t[1], v[i:i + 1]))
        for h in range(Hq):
            p = torch.softmax(kk[:, h // (Hq // Hkv)] @ q[i, h] * D ** -0.5, 0)
            out[i, h] = p @ vv[:, h // (Hq // Hkv)]
    o = out.view(B, -1) @ dense(b.wo).T
    return o, rms(resid.double() + o, b.moe_norm)


def test_sequences_begin_run_and_end(cuda_device):
    cfg, page, shared, B = inputs.TINY, 16, 48, 4
    b = decode_block.SharedBlock(cfg, 4, 2, 64, batch=B, capacity=112, shared=shared, page=page, device=cuda_device, group=64,
                                 groups=4, top_groups=2)
    b.k_cache.normal_()
    b.v_cache.normal_()
    b.bias.copy_(torch.randn(cfg.E, generator=torch.Generator().manual_seed(1)) * 0.02)
    pool = b.k_cache.shape[0] - b.shared.numel()
    prefix = tuple(c[b.shared.long()].flatten(0, 1).double() for c in (b.k_cache, b.v_cache))
    none = tuple(c[:0] for c in prefix)
    tokens = [None] * B
    gate, up, down = (mx(m) for m in b.experts)
    resid = torch.randn(B, cfg.d, device=cuda_device)
    seen, layer, graph = [], moe.layer, None

    def begin(i, shares):
        b.begin(i, shares)
        tokens[i] = prefix if shares else none

    try:
        decode_block.moe.layer = lambda x, ids, w, *e, **kw: (seen.append((x, ids, w)), layer(x, ids, w, *e, **kw))[1]
        for step in range(44):
            if step in (0, 3, 5):
                begin({0: 0, 3: 1, 5: 2}[step], step != 3)
            if step == 24:
                b.end(0)
                tokens[0] = None
            if step == 27:
                begin(3, True)
                begin(0, False)
            before = resid.clone()
            o, x_ref = reference(b, before, tokens)
            if step < 2:
                b.step(resid)
            else:
                if graph is None:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):     # (records, does not run)
                        b.step(resid)
                graph.replay()
            torch.cuda.synchronize()
            run = [i for i in range(B) if tokens[i] is not None]
            for i in run:   # what the step has appended, from the cache, at the place that the table names
                n = len(tokens[i][0])
                pg, row = int(b.table[i, n // page]), n % page
                tokens[i] = tuple(torch.cat((t, c[pg, row][None].double())) for t, c in zip(tokens[i], (b.k_cache, b.v_cache)))
            assert b.lens.tolist() == [0 if t is None else len(t[0]) for t in tokens], step
            used = [int(b.table[i, j]) for i in run
                    for j in range(shared // page if bool(b.shares[i]) else 0, -(-len(tokens[i][0]) // page))]
            left = b.free[:int(b.n_free)].tolist()
            assert len(set(used + left)) == len(used) + len(left) == pool, f"step {step}: a page lost or held twice"
            x, ids, w = seen[-1]
            err = (x.double() - x_ref)[run].norm() / x_ref[run].norm()
            assert err <= 10 * 2.0 ** -8, f"step {step}: the expert layer's input is {err:.3g} off"
            # the router's choice from the layer's own input
            p = torch.softmax(x.double() @ b.router.double().T, -1)
            key = (p + b.bias.double()).view(B, 4, -1)
            top = key.sort(-1, descending=True)[0][..., :2].sum(-1).sort(-1, descending=True)[1][:, :2]
            for i in run:
                for e, we in zip(ids[i].tolist(), w[i].tolist()):
                    assert e // (cfg.E // 4) in top[i].tolist()
                    assert abs(we - float(p[i, e] / p[i, ids[i].long()].sum())) <= 1e-4
            xd = x.double()
            y = torch.zeros_like(xd)
            for i in run:
                for e, we in zip(ids[i].tolist(), w[i].double().tolist()):
                    g, u = gate[e] @ xd[i], up[e] @ xd[i]
                    y[i] += we * (down[e] @ (g * torch.sigmoid(g) * u))
            want = (o + y)[run]
            err = ((resid.double() - before.double())[run] - want).norm() / want.norm()
            assert err <= 10 * 2.0 ** -8, f"step {step}: the update is {err:.3g} off"
    finally:
        decode_block.moe.layer = layer
    assert moe.device_error(cuda_device) == 0


def test_example_runs_with_a_shared_prefix(cuda_device, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["decode_block.py", "--batch", "3", "--shared", "256", "--steps", "4"])
    decode_block.main()
    assert "lengths now" in capsys.readouterr().out
