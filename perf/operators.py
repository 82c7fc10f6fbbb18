"""What the operators of the decode block around the expert layer are measured on.

paged_attention, rope_append, norm_residual and matvec4, each as a plain form
(elementary torch operations, 32 bits inside, 64 for rotary angles), as the
package's call (where `own` is true) and as a definition in 64 bits (`exact`).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
E4M3_MAX = 448.0


def listed():
    return [
        # one user, a short chat: latency (the head layout of a Qwen3-style block)
        {"name": "attn_single", "op": "attn", "B": 1, "Hq": 32, "Hkv": 4, "D": 128, "page": 16, "max_len": 777,
         "lens": "full", "window": 0, "sinks": 0, "dtype": "bf16", "cache": "bf16"},
        # continuous batching: 32 users at very different lengths, one of them not begun
        {"name": "attn_ragged", "op": "attn", "B": 32, "Hq": 32, "Hkv": 4, "D": 128, "page": 64, "max_len": 32768,
         "lens": "log", "window": 0, "sinks": 0, "dtype": "bf16", "cache": "bf16"},
        # a few users with whole books in the context, 8-bit cache
        {"name": "attn_long_e4m3", "op": "attn", "B": 4, "Hq": 64, "Hkv": 8, "D": 128, "page": 128, "max_len": 131072,
         "lens": "full", "window": 0, "sinks": 0, "dtype": "fp16", "cache": "e4m3"},
        # streaming: a sliding window and a few first tokens that stay visible
        {"name": "attn_window", "op": "attn", "B": 64, "Hq": 16, "Hkv": 2, "D": 64, "page": 32, "max_len": 20000,
         "lens": "log", "window": 1000, "sinks": 4, "dtype": "fp16", "cache": "fp16"},
        # a small model with a key-value head for each head, odd sizes throughout
        {"name": "attn_heads_odd", "op": "attn", "B": 7, "Hq": 12, "Hkv": 12, "D": 80, "page": 24, "max_len": 5003,
         "lens": "full", "window": 0, "sinks": 0, "dtype": "bf16", "cache": "bf16"},
        # one decode step of 32 users, 8-bit cache
        {"name": "rope_decode", "op": "rope", "T": 32, "Hq": 32, "Hkv": 4, "D": 128, "rot": 128, "interleaved": False,
         "page": 64, "pages": 96, "scaling": "none", "max_pos": 32768, "dtype": "bf16", "cache": "e4m3"},
        # a long prompt written at once: interleaved pairs, half of the head, scaled for a long context
        {"name": "rope_prompt", "op": "rope", "T": 16384, "Hq": 64, "Hkv": 8, "D": 128, "rot": 64, "interleaved": True,
         "page": 128, "pages": 160, "scaling": "by_parts", "max_pos": 1000000, "dtype": "bf16", "cache": "bf16"},
        # one token between two blocks: residual add and the next block's norm
        {"name": "norm_single", "op": "norm", "T": 1, "d": 2048, "kind": "rms", "post": False, "gate": "none", "act": "none",
         "alpha": 1.0, "dtype": "bf16", "resid": "bf16"},
        # a prompt through the widest form: norms on both sides, a gate, a 32-bit residual
        {"name": "norm_prompt", "op": "norm", "T": 8192, "d": 7168, "kind": "rms", "post": True, "gate": "full",
         "act": "sigmoid", "alpha": 0.5, "dtype": "bf16", "resid": "fp32"},
        # one token's query projection of a Qwen3-style block (32 heads of 128 from 2048)
        {"name": "matvec_single", "op": "matvec", "T": 1, "N": 4096, "K": 2048, "group": 128, "zeros": False,
         "dtype": "bf16"},
        # one token through a wide dense projection: the weights' bytes count
        {"name": "matvec_wide", "op": "matvec", "T": 1, "N": 28672, "K": 8192, "group": 64, "zeros": True,
         "dtype": "bf16"},
        # 16 users share one read of the weights; an odd number of rows, the smallest groups
        {"name": "matvec_batch", "op": "matvec", "T": 16, "N": 7169, "K": 4096, "group": 32, "zeros": True,
         "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "norm", "matvec"])
    dt = rng.choice(["bf16", "fp16"])
    if op == "attn":
        Hq, Hkv = rng.choice([(32, 4), (16, 2), (64, 8), (8, 8), (12, 12), (20, 1), (40, 8), (9, 3)])
        D = rng.choice([64, 80, 128, 128, 192, 256])
        B = _log(rng, 1, 64)
        most = min(131072, 200_000_000 // (B * Hkv * D), 16_000_000 // (B * Hq))
        win = rng.random() < 0.4
        return {"op": "attn", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "page": rng.choice([8, 16, 24, 32, 64, 128]),
                "max_len": _log(rng, 1, most), "lens": rng.choice(["full", "log"]),
                "window": _log(rng, 1, 8192) if win else 0, "sinks": rng.randint(0, 64) if win else 0,
                "dtype": dt, "cache": rng.choice([dt, dt, "e4m3"])}
    if op == "rope":
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 3, 4, 8])
        D = rng.choice([64, 80, 128, 256])
        cache = rng.choice([dt, dt, "e4m3"])
        T = _log(rng, 1, 3000 * 8 * 128 // (Hkv * D) if cache == "e4m3" else 16384 * 8 * 128 // (max(Hkv, Hq // 8) * D))
        page = rng.choice([8, 16, 24, 64, 128])
        return {"op": "rope", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rng.choice([D, D // 2, D // 4]),
                "interleaved": rng.random() < 0.5, "page": page, "pages": -(-T * 5 // (4 * page)) + 1,
                "scaling": rng.choice(["none", "by_parts"]), "max_pos": _log(rng, 4096, 1000000), "dtype": dt,
                "cache": cache}
    if op == "norm":
        d = _log(rng, 64, 8192)
        d = d if rng.random() < 0.3 else max(64, d // 64 * 64)
        return {"op": "norm", "T": _log(rng, 1, 58_000_000 // d), "d": d, "kind": rng.choice(["rms", "layer"]),
                "post": rng.random() < 0.5, "gate": rng.choice(["none", "full", "row", "column"]),
                "act": rng.choice(["none", "sigmoid"]), "alpha": rng.choice([1.0, 0.25]), "dtype": dt,
                "resid": rng.choice([dt, "fp32"])}
    N, K, T = _log(rng, 100, 28672), 128 * _log(rng, 2, 64), rng.choice([1, 1, 2, 5, 8, 16])
    return {"op": "matvec", "T": T, "N": N if rng.random() < 0.5 else max(64, N // 64 * 64), "K": K,
            "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5, "dtype": dt}


def _lengths(case, g):
    B, most = case["B"], case["max_len"]
    u = torch.rand(B, generator=g, dtype=torch.float64)
    if case["lens"] == "full":
        return (most * (1 - 0.1 * u)).long().clamp(min=1)
    lens = torch.exp(u * math.log(most)).long().clamp(1, most)
    lens[0] = most
    if B > 2:
        lens[B // 2] = 0
    return lens


def _inv_freq(case):
    """Radians a position for each pair; by_parts: low frequencies divided by 8, high ones kept, a ramp between
    1 and 32 turns within the 4096 positions of the original context."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "by_parts":
        ramp = ((4096 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = f * (ramp + (1 - ramp) / 8)
    return f


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator(device="cuda").manual_seed(seed + 1)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gg, device="cuda", dtype=dt if dtype != torch.float32 else dtype)
                * std).to(dtype)

    s = {"case": case}
    if case["op"] == "attn":
        B, Hkv, D, P = case["B"], case["Hkv"], case["D"], case["page"]
        lens = _lengths(case, g)
        used = (lens + P - 1) // P
        most = max(1, int(used.max()))
        pages = int(used.sum()) + 3
        order = torch.randperm(pages, generator=g)
        table = torch.zeros(B, most, dtype=torch.int64)
        begin = torch.cumsum(used, 0) - used
        at = torch.arange(most)
        inside = at[None, :] < used[:, None]
        table[inside] = order[(begin[:, None] + at[None, :])[inside]]
        cdt = DTYPES[case["cache"]]
        s["q"] = randn(B, case["Hq"], D, std=2.0)
        s["k_scale"], s["v_scale"] = (0.03125, 0.0234375) if case["cache"] == "e4m3" else (1.0, 1.0)
        s["k"] = randn(pages, P, Hkv, D, std=1 / s["k_scale"], dtype=cdt)
        s["v"] = randn(pages, P, Hkv, D, std=1 / s["v_scale"], dtype=cdt)
        s["table"] = table.int().cuda()
        s["lens"] = lens.int().cuda()
        s["scale"] = D ** -0.5
        # the joins' scratch, which a user's program makes once and keeps
        s["ws"] = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")
    elif case["op"] == "rope":
        T, Hkv, D = case["T"], case["Hkv"], case["D"]
        # one projection's output holds the query, key and value heads of each token side by side
        qkv = randn(T, case["Hq"] + 2 * Hkv, D)
        s["q"], s["kn"], s["vn"] = qkv.split([case["Hq"], Hkv, Hkv], dim=1)
        cdt = DTYPES[case["cache"]]
        s["k_scale"], s["v_scale"] = (0.03125, 0.0234375) if case["cache"] == "e4m3" else (1.0, 1.0)
        s["k"] = randn(case["pages"], case["page"], Hkv, D, dtype=cdt)
        s["v"] = randn(case["pages"], case["page"], Hkv, D, dtype=cdt)
        s["slots"] = torch.randperm(case["pages"] * case["page"], generator=g)[:T].cuda()
        s["pos"] = torch.randint(0, case["max_pos"], (T,), generator=g).int().cuda()
        s["freqs"] = _inv_freq(case).cuda()
        s["mscale"] = 1.0 if case["scaling"] == "none" else 0.1 * math.log(8) + 1
    elif case["op"] == "norm":
        T, d = case["T"], case["d"]
        s["y"] = randn(T, d)
        s["r"] = randn(T, d, std=4.0, dtype=DTYPES[case["resid"]])
        s["gate"] = {"none": None, "full": (T, d), "row": (T, 1), "column": (1, d)}[case["gate"]]
        if s["gate"] is not None:
            s["gate"] = randn(*s["gate"])
        bias = case["kind"] == "layer"
        s["post"] = (1 + randn(d, std=0.1), randn(d, std=0.1) if bias else None) if case["post"] else None
        s["pre"] = (1 + randn(d, std=0.1), randn(d, std=0.1) if bias else None)
    else:
        T, N, K, G = case["T"], case["N"], case["K"], case["group"]
        s["x"] = randn(T, K)
        s["codes"] = torch.randint(0, 256, (N, K // 2), generator=gg, device="cuda", dtype=torch.uint8)
        s["scales"] = (0.01 * (0.5 + torch.rand(N, K // G, generator=gg, device="cuda"))).to(dt)
        s["zeros"] = torch.randint(0, 16, (N, K // G), generator=gg, device="cuda", dtype=torch.uint8) \
            if case["zeros"] else None
    return s


def _rotated(x, cos, sin, rot, interleaved):
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        p, q = a[..., 0::2], a[..., 1::2]
        a = torch.stack((p * cos - q * sin, q * cos + p * sin), -1).flatten(-2)
    else:
        p, q = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat((p * cos - q * sin, q * cos + p * sin), -1)
    return torch.cat((a, rest), -1)


def _normed(x, spec, kind):
    w, b = spec
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.to(x.dtype)
    return x if b is None else x + b.to(x.dtype)


def _to_cache(x, scale, dtype):
    if dtype != torch.float8_e4m3fn:
        return x.to(dtype)
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(dtype)


def _put(cache, slots, rows):
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    raw.view(-1, *cache.shape[2:])[slots] = rows.view(raw.dtype)


def _attn_plain(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    at = s["table"].long()
    k = s["k"][at].flatten(1, 2).float() * s["k_scale"]
    v = s["v"][at].flatten(1, 2).float() * s["v_scale"]
    L = k.shape[1]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    j, n = torch.arange(L, device="cuda")[None, :], s["lens"].long()[:, None]
    seen = j < n
    if c["window"]:
        seen &= (j >= n - c["window"]) | (j < c["sinks"])
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(score - m)
    l = p.sum(-1, keepdim=True)
    v = v * (j < n)[:, :, None, None]
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(l > 0, l, torch.ones_like(l))
    return o.view(B, Hq, D).to(s["q"].dtype), (m + torch.log(l)).view(B, Hq)


def _rope_plain(s):
    c = s["case"]
    ang = s["pos"].double()[:, None, None] * s["freqs"]
    cos, sin = (ang.cos() * s["mscale"]).float(), (ang.sin() * s["mscale"]).float()
    q = _rotated(s["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
    kn = _rotated(s["kn"].float(), cos, sin, c["rot"], c["interleaved"])
    _put(s["k"], s["slots"], _to_cache(kn, s["k_scale"], s["k"].dtype))
    _put(s["v"], s["slots"], _to_cache(s["vn"].float(), s["v_scale"], s["v"].dtype))
    return q, s["k"], s["v"]


def _norm_plain(s):
    c = s["case"]
    u = s["y"].float()
    if s["post"] is not None:
        u = _normed(u, s["post"], c["kind"])
    if s["gate"] is not None:
        g = s["gate"].float()
        u = u * (1 / (1 + torch.exp(-g)) if c["act"] == "sigmoid" else g)
    r = s["r"].float() + c["alpha"] * u
    return r.to(s["r"].dtype), _normed(r, s["pre"], c["kind"]).to(s["y"].dtype)


def _weights(s, dtype):
    c = s["case"]
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(c["N"], -1, c["group"]).to(dtype)
    zero = 8 if s["zeros"] is None else s["zeros"].to(dtype)[:, :, None]
    return ((codes - zero) * s["scales"].to(dtype)[:, :, None]).view(c["N"], c["K"])


def run(state):
    s = state
    c = s["case"]
    if not own:
        if c["op"] == "attn":
            return _attn_plain(s)
        if c["op"] == "rope":
            return _rope_plain(s)
        if c["op"] == "norm":
            return _norm_plain(s)
        return torch.matmul(s["x"].float(), _weights(s, torch.float32).T).to(s["x"].dtype)
    import mixture_experts_decode_gb300 as moe
    if c["op"] == "attn":
        return moe.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=s["scale"], window=c["window"],
                                   sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"], workspace=s["ws"],
                                   return_lse=True)
    if c["op"] == "rope":
        q = moe.rope_append(s["q"], s["kn"], s["vn"], s["pos"], s["slots"], s["freqs"], s["k"], s["v"],
                            interleaved=c["interleaved"], mscale=s["mscale"], k_scale=s["k_scale"],
                            v_scale=s["v_scale"])
        return q, s["k"], s["v"]
    if c["op"] == "norm":
        spec = lambda n: None if n is None else moe.Norm(n[0], n[1], eps=1e-6, kind=c["kind"])  # noqa: E731
        return moe.norm_residual(s["y"], s["r"], post=spec(s["post"]), gate=s["gate"], gate_act=c["act"],
                                 alpha=c["alpha"], pre=spec(s["pre"]))
    return moe.matvec4(s["x"], moe.W4(s["codes"], s["scales"], s["zeros"]))


def _seen(case, lens):
    if not case["window"]:
        return lens
    return torch.minimum(lens, torch.clamp(lens, max=case["window"]) + case["sinks"])


def work(case):
    if case["op"] == "attn":
        # the expected length stands for the seeds' own
        n, most = case["B"], case["max_len"]
        if case["lens"] == "full":
            lens = torch.full((n,), most * 0.95, dtype=torch.float64).clamp(min=1)
        else:
            lens = torch.exp((torch.arange(n, dtype=torch.float64) + 0.5) / n * math.log(most)).clamp(1, most)
            lens[0] = most
        seen = float(_seen(case, lens).sum())
        per = case["Hkv"] * case["D"]
        return {"bytes": 2 * seen * per * SIZES[case["cache"]] + 2 * n * case["Hq"] * case["D"] * 2 + 4 * n * case["Hq"],
                "flops": 4 * seen * case["Hq"] * case["D"]}
    if case["op"] == "rope":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        return {"bytes": T * D * (4 * Hq + 2 * Hkv * (2 + SIZES[case["cache"]])) + 12 * T,
                "flops": 3 * T * case["rot"] * (Hq + Hkv)}
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        gate = {"none": 0, "full": T * d, "row": T, "column": d}[case["gate"]]
        return {"bytes": T * d * (4 + 2 * SIZES[case["resid"]]) + 2 * gate, "flops": T * d * (16 if case["post"] else 8)}
    T, N, K, G = case["T"], case["N"], case["K"], case["group"]
    return {"bytes": N * K // 2 + N * (K // G) * (3 if case["zeros"] else 2) + 2 * T * (K + N), "flops": 2 * T * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        B, Hq, Hkv, D, P = case["B"], case["Hq"], case["Hkv"], case["D"], case["page"]
        out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            j = [t for t in range(n) if not case["window"] or t >= n - case["window"] or t < case["sinks"]]
            if not j:
                continue
            j = torch.tensor(j, device="cuda")
            page, off = s["table"][b].long()[j // P], j % P
            for h in range(Hkv):
                k = s["k"][page, off, h].double() * s["k_scale"]
                v = s["v"][page, off, h].double() * s["v_scale"]
                heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                score = s["q"][b, heads].double() @ k.T * s["scale"]
                lse[b, heads] = torch.logsumexp(score, -1)
                out[b, heads] = torch.softmax(score, -1) @ v
        return out, lse
    if case["op"] == "rope":
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * s["freqs"][None, :])[:, None, :] * s["mscale"]
        rot = case["rot"]

        def rotate(x):
            x = x.double().clone()
            a = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(x[..., a[0]], x[..., a[1]]) * turn
            x[..., a[0]], x[..., a[1]] = z.real, z.imag
            return x

        k, v = s["k"].double(), s["v"].double()
        top = E4M3_MAX if case["cache"] == "e4m3" else math.inf
        k.view(-1, *k.shape[2:])[s["slots"]] = (rotate(s["kn"]) / s["k_scale"]).clamp(-top, top)
        v.view(-1, *v.shape[2:])[s["slots"]] = (s["vn"].double() / s["v_scale"]).clamp(-top, top)
        return rotate(s["q"]), k, v
    if case["op"] == "norm":
        def norm(x, spec):
            if case["kind"] == "layer":
                var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
            else:
                var, mean = x.square().mean(-1, keepdim=True), 0.0
            x = (x - mean) * torch.rsqrt(var + 1e-6) * spec[0].double()
            return x if spec[1] is None else x + spec[1].double()

        u = s["y"].double() if s["post"] is None else norm(s["y"].double(), s["post"])
        if s["gate"] is not None:
            u = u * (torch.sigmoid(s["gate"].double()) if case["act"] == "sigmoid" else s["gate"].double())
        r = torch.add(s["r"].double(), u, alpha=case["alpha"])
        return r, norm(r, s["pre"])
    w = torch.empty(case["N"], case["K"], dtype=torch.float64, device="cuda")
    w[:, 0::2], w[:, 1::2] = (s["codes"] % 16).double(), (s["codes"] // 16).double()
    z = torch.full_like(s["scales"], 8, dtype=torch.float64) if s["zeros"] is None else s["zeros"].double()
    w -= z.repeat_interleave(case["group"], 1)
    w *= s["scales"].double().repeat_interleave(case["group"], 1)
    return s["x"].double() @ w.T
