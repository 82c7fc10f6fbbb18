"""64-bit references and bounds of the decode block's operators (not collected by pytest)."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -23   # twice FP32's half step: covers sums that truncate


def half_step(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2


def visible(n: int, window: int, sinks: int):
    return [j for j in range(n) if window == 0 or j >= n - window or j < sinks]


def attention(q, k, v, table, lens, scale, window=0, sinks=0, k_scale=1.0, v_scale=1.0):
    """(out, lse, out_bound, lse_bound) in float64; a token of a page outside the cache is left out.

    Bounds: the output's own rounding, plus sum p|v| times the relative error
    of the weights: p as two 16-bit values (2^-17), exp2 (2^-20 in all), the
    scores' FP32 dots (2 * D terms of S = the largest scale * sum |q k|) and
    the FP32 sums over the keys."""
    B, Hq, D = q.shape
    pages, P, Hkv, _ = k.shape
    G = Hq // Hkv
    dev = q.device
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=dev)
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    tab = table.cpu()
    for b, n in enumerate(lens.cpu().tolist()):
        rows = [(int(tab[b, j // P]), j % P) for j in visible(max(0, min(n, tab.shape[1] * P)), window, sinks)]
        rows = [r for r in rows if 0 <= r[0] < pages]
        if not rows:
            continue
        pg = torch.tensor([r[0] for r in rows], device=dev)
        of = torch.tensor([r[1] for r in rows], device=dev)
        kk = k[pg, of].double() * k_scale      # [n, Hkv, D]
        vv = v[pg, of].double() * v_scale
        for h in range(Hq):
            a, w = kk[:, h // G], vv[:, h // G]
            x = q[b, h].double()
            s = a @ x * scale
            S = float((a.abs() @ x.abs()).max() * abs(scale))
            p = torch.softmax(s, 0)
            out[b, h] = p @ w
            lse[b, h] = torch.logsumexp(s, 0)
            rel = 2 * D * U32 * S + len(rows) * U32
            ob[b, h] = half_step(q.dtype) * out[b, h].abs() + (p @ w.abs()) * (2.0 ** -17 + 2.0 ** -20 + rel) \
                + (2.0 ** -24 if q.dtype == torch.float16 else 0.0)
            lb[b, h] = rel + 2.0 ** -20 + lse[b, h].abs() * U32
    return out, lse, ob, lb


def rotate(x, pos, freqs, rot, interleaved, mscale):
    """(rotated, size of the terms) in float64 for x [T, H, D]."""
    x = x.double()
    a = pos.double()[:, None] * freqs.double()[None, :]
    c, s = (a.cos() * mscale)[:, None], (a.sin() * mscale)[:, None]
    i0 = torch.arange(0, rot, 2, device=x.device) if interleaved else torch.arange(rot // 2, device=x.device)
    i1 = i0 + 1 if interleaved else i0 + rot // 2
    out, size = x.clone(), torch.zeros_like(x)
    u, w = x[..., i0], x[..., i1]
    out[..., i0], out[..., i1] = u * c - w * s, w * c + u * s
    size[..., i0] = size[..., i1] = (u.abs() + w.abs()) * mscale
    return out, size


def norm(v, w, b, eps, kind):
    """(normed, bound of FP32's error) in float64.  Each thread adds at most 64
    squares and a row's threads join in ten steps: (64 + 10) half steps on the
    mean and on the mean square (2^-17 together with the products), relative
    to the row's largest value."""
    v = v.double()
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    c = v - mean
    inv = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    wd = torch.ones_like(v[0]) if w is None else w.double()
    bd = torch.zeros_like(v[0]) if b is None else b.double()
    return c * inv * wd + bd, 2.0 ** -16 * (v.abs().amax(-1, keepdim=True) * inv * wd.abs() + bd.abs())


def norm_residual(y, r, post, gate, act, alpha, pre):
    """((r', bound), (x, bound)) in float64; post, pre = (w, b, eps, kind) or None."""
    u, err = y.double(), torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    if post is not None:
        u, err = norm(u, *post)
    if gate is not None:
        g = torch.sigmoid(gate.double()) if act == "sigmoid" else gate.double()
        u, err = u * g, err * g.abs() + 8 * U32 * (u * g).abs()
    rr = (0.0 if r is None else r.double()) + alpha * u
    rerr = err * abs(alpha) + 4 * U32 * ((0.0 if r is None else r.double().abs()) + (alpha * u).abs())
    if pre is None:
        return (rr, rerr), (rr, rerr)
    x, xerr = norm(rr, *pre)
    c = rr - (rr.mean(-1, keepdim=True) if pre[3] == "layer" else 0.0)
    inv = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + pre[2])
    wd = torch.ones_like(rr[0]) if pre[0] is None else pre[0].double()
    # an error e of r' moves x by at most about |w| inv (2 max e + |x / w| ...)
    xerr = xerr + 4 * rerr.amax(-1, keepdim=True) * inv * wd.abs() * (1 + (c * inv).abs())
    return (rr, rerr), (x, xerr)


def matvec4(x, codes, scales, zeros, group):
    """(y, bound of FP32's error) in float64: products of 16 + c, exact, in
    chains of at most `group` terms, joined over K / group groups."""
    N, half = codes.shape
    K = 2 * half
    c = torch.empty(N, K, dtype=torch.float64, device=x.device)
    c[:, 0::2], c[:, 1::2] = (codes & 15).double(), (codes >> 4).double()
    z = torch.full_like(scales, 8, dtype=torch.float64) if zeros is None else zeros.double()
    z, s = z.repeat_interleave(group, 1), scales.double().repeat_interleave(group, 1)
    xd = x.double()
    y = xd @ ((c - z) * s).T
    size = xd.abs() @ ((32 + c + z) * s.abs()).T
    return y, size * U32 * (group + K // group + 8)
