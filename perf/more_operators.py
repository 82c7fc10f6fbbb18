"""What the operators of a serving step around the decode block are measured on.

shared_prefix_attention (a batch whose sequences begin with the same long
prefix), router_grouped_topk (scores, a balancing bias, groups of experts),
plan_pages and release_pages (block tables, slots and positions on the device
from the requests' lengths), each as a plain form (elementary torch operations,
32 bits inside, 64 for the router's borders), as the package's call (where
`own` is true) and as a definition in 64 bits (`exact`).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def listed():
    return [
        # four users behind a short instruction, their first words
        {"name": "prefix_short", "op": "attn", "B": 4, "Hq": 32, "Hkv": 4, "D": 128, "page": 16, "prefix_pages": 40,
         "max_own": 60, "others": False, "dtype": "bf16", "cache": "bf16"},
        # 32 users of one assistant: a long system prompt with its tools, chats of different lengths, some users elsewhere
        {"name": "prefix_chat", "op": "attn", "B": 32, "Hq": 32, "Hkv": 4, "D": 128, "page": 64, "prefix_pages": 128,
         "max_own": 1500, "others": True, "dtype": "bf16", "cache": "bf16"},
        # 64 questions about one book, 8-bit cache
        {"name": "prefix_book_e4m3", "op": "attn", "B": 64, "Hq": 64, "Hkv": 8, "D": 128, "page": 128,
         "prefix_pages": 512, "max_own": 700, "others": False, "dtype": "bf16", "cache": "e4m3"},
        # 300 samples drawn from one prompt: many rows a key
        {"name": "prefix_samples", "op": "attn", "B": 300, "Hq": 16, "Hkv": 2, "D": 64, "page": 32, "prefix_pages": 300,
         "max_own": 400, "others": False, "dtype": "fp16", "cache": "fp16"},
        # a key-value head for each head, odd sizes throughout
        {"name": "prefix_odd", "op": "attn", "B": 7, "Hq": 12, "Hkv": 12, "D": 80, "page": 24, "prefix_pages": 209,
         "max_own": 333, "others": True, "dtype": "fp16", "cache": "e4m3"},
        # one token of a Qwen3-style layer's router with a balancing bias
        {"name": "router_single", "op": "router", "T": 1, "E": 128, "k": 8, "score": "softmax", "bias": True, "groups": 1,
         "top_groups": 1, "group_score": "max", "renorm": True, "scale": 1.0, "dtype": "fp32"},
        # one decode step of 33 users through a DeepSeek-V3-style gate: 4 of 8 groups, sigmoid
        {"name": "router_step", "op": "router", "T": 33, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "dtype": "fp32"},
        # the same gate on the tokens of long prompts
        {"name": "router_prompts", "op": "router", "T": 65536, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "dtype": "fp32"},
        # a decode step of 64 running requests, one token each
        {"name": "plan_step", "op": "plan", "B": 64, "page": 64, "max_pages": 512, "max_past": 30000, "max_new": 1,
         "begin": 0.0, "shared": 0, "room": 1.1},
        # prompts of many requests that begin behind a shared prefix, beside running ones
        {"name": "plan_prompts", "op": "plan", "B": 500, "page": 16, "max_pages": 2048, "max_past": 20000, "max_new": 8000,
         "begin": 0.4, "shared": 100, "room": 1.2},
        # a few requests of a batch end
        {"name": "release_few", "op": "release", "B": 64, "page": 64, "max_pages": 512, "max_past": 30000, "ends": 0.1,
         "shared": 20},
        # most of a large batch of long requests ends
        {"name": "release_many", "op": "release", "B": 1000, "page": 16, "max_pages": 4096, "max_past": 65000, "ends": 0.9,
         "shared": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "router", "router", "plan", "release"])
    if op == "attn":
        dt = rng.choice(["bf16", "fp16"])
        Hq, Hkv = rng.choice([(32, 4), (16, 2), (64, 8), (8, 8), (12, 12), (20, 1), (40, 8), (9, 3)])
        D = rng.choice([64, 80, 128, 128, 192, 256])
        B = _log(rng, 2, 300)
        page = rng.choice([8, 16, 24, 32, 64, 128])
        most = min(65536, 120_000_000 // (B * Hq), 67_000_000 // (Hkv * D))
        return {"op": "attn", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
                "prefix_pages": max(1, _log(rng, page, most) // page),
                "max_own": _log(rng, 1, max(1, min(2000, 30_000_000 // (B * Hkv * D), 8_000_000 // (B * Hq)))),
                "others": rng.random() < 0.4, "dtype": dt, "cache": rng.choice([dt, dt, "e4m3"])}
    if op == "router":
        E = rng.choice([8, 16, 64, 96, 128, 160, 256, 256, 320, 512])
        groups = rng.choice([g for g in (1, 1, 2, 4, 5, 8, 16) if E % g == 0 and E // g >= 2])
        top = rng.randint(1, groups)
        return {"op": "router", "T": _log(rng, 1, 16_000_000 // E if E >= 256 else 65536), "E": E,
                "k": min(rng.choice([1, 2, 4, 6, 8, 8]), top * (E // groups)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.7, "groups": groups,
                "top_groups": top, "group_score": rng.choice(["max", "top2"]), "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["fp32", "fp32", "bf16", "fp16"])}
    B, page = _log(rng, 1, 1000), rng.choice([8, 16, 24, 64, 128])
    most = _log(rng, 100, min(60000, (1_000_000 if op == "plan" else 4_000_000) // B * page))
    c = {"op": op, "B": B, "page": page, "max_past": most, "shared": rng.choice([0, most // page // 4])}
    if op == "release":
        return dict(c, max_pages=-(-most // page) + rng.randint(1, 70), ends=rng.choice([0.1, 0.5, 1.0]))
    new = 1 if rng.random() < 0.4 else _log(rng, 2, min(8000, 1_500_000 // B))
    return dict(c, max_pages=-(-(most + new) // page) + rng.randint(0, 70), max_new=new,
                begin=0.0 if new == 1 else rng.choice([0.2, 0.5, 1.0]), room=rng.choice([1.1, 1.1, 0.9]))


def _randn(gg, dtype, *shape, std=1.0):
    return (torch.randn(*shape, generator=gg, device="cuda") * std).to(dtype)


def _tokens(case):
    """Rows of the plan's outputs: what the step may hold, a tenth above what its requests are expected to bring."""
    B, new = case["B"], case["max_new"]
    return B if new == 1 else max(1, math.ceil(B * case["begin"] * new * 0.55 + B + new))


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator(device="cuda").manual_seed(seed + 1)
    s = {"case": case}
    if case["op"] == "attn":
        B, Hkv, D, P = case["B"], case["Hkv"], case["D"], case["page"]
        dt, cdt = DTYPES[case["dtype"]], DTYPES[case["cache"]]
        ns, most = case["prefix_pages"], case["max_own"]
        mine = (most * torch.rand(B, generator=g) ** 2).long().clamp(min=1, max=most)
        mine[0] = most
        shares = torch.ones(B, dtype=torch.bool)
        if case["others"]:
            shares[3::5] = False
            mine[B // 2] = 0
        lens = torch.where(shares, ns * P + mine, mine)
        used = (mine + P - 1) // P
        pages = int(used.sum()) + ns + 3
        order = torch.randperm(pages, generator=g)
        s["shared"] = order[:ns].int().cuda()
        table = torch.zeros(B, ns + -(-most // P), dtype=torch.int64)
        table[shares, :ns] = order[:ns]
        at = torch.arange(table.shape[1])
        first = torch.where(shares, ns, 0)
        inside = (at[None, :] >= first[:, None]) & (at[None, :] < (first + used)[:, None])
        begin = torch.cumsum(used, 0) - used + ns
        table[inside] = order[(begin[:, None] + at[None, :] - first[:, None])[inside]]
        s["q"] = _randn(gg, dt, B, case["Hq"], D, std=2.0)
        s["k_scale"], s["v_scale"] = (0.03125, 0.0234375) if case["cache"] == "e4m3" else (1.0, 1.0)
        s["k"] = _randn(gg, cdt, pages, P, Hkv, D, std=1 / s["k_scale"])
        s["v"] = _randn(gg, cdt, pages, P, Hkv, D, std=1 / s["v_scale"])
        s["table"], s["lens"] = table.int().cuda(), lens.int().cuda()
        s["shares"] = shares.cuda() if case["others"] else None
        s["scale"] = D ** -0.5
        # the pieces' scratch, which a user's program makes once and keeps
        if own:
            import mixture_experts_decode_gb300 as moe
            s["ws"] = moe.shared_prefix_workspace(B, case["Hq"], Hkv, D)
    elif case["op"] == "router":
        T, E = case["T"], case["E"]
        s["logits"] = _randn(gg, DTYPES[case["dtype"]], T, E)
        # sigmoid scores lie in 0..1, softmax ones around 1 / E
        s["bias"] = _randn(gg, torch.float32, E, std=0.1 if case["score"] == "sigmoid" else 0.2 / E) \
            if case["bias"] else None
    else:
        B, P, ns, most = case["B"], case["page"], case["shared"], case["max_past"]
        past = torch.exp(torch.rand(B, generator=g, dtype=torch.float64) * math.log(most)).long().clamp(1, most)
        shares = torch.rand(B, generator=g) < 0.8
        if ns:
            past = torch.where(shares, past.clamp(min=ns * P), past)
        if case["op"] == "plan":
            new = torch.ones(B, dtype=torch.int64)
            fresh = torch.rand(B, generator=g) < case["begin"]
            if case["max_new"] > 1:
                new = torch.where(fresh, (torch.rand(B, generator=g) * case["max_new"]).long() + 1, new)
            past = torch.where(fresh, torch.where(shares, ns * P, 0), past)
            if B > 3:
                new[B // 3] = 0  # a request that waits
            s["new"] = new.int().cuda()
        else:
            s["ended"] = (torch.rand(B, generator=g) < case["ends"]).cuda()
            new = torch.zeros(B, dtype=torch.int64)
        have = (past + P - 1) // P
        need = int(((past + new + P - 1) // P - have).sum())
        pages = int(have.sum()) + math.ceil(need * case.get("room", 0)) + ns + 8
        order = torch.randperm(pages, generator=g)
        table = torch.full((B, case["max_pages"]), -1, dtype=torch.int64)
        at = torch.arange(case["max_pages"])
        inside = at[None, :] < have[:, None]
        begin = torch.cumsum(have, 0) - have + ns
        table[inside] = order[(begin[:, None] + at[None, :])[inside]]
        if ns:
            n0 = min(ns, case["max_pages"])
            held = shares[:, None] & (at[None, :] < n0) & inside
            table[held] = order[at.expand(B, -1)[held]]
        s["shared"] = order[:ns].int().cuda()
        s["shares"] = shares.cuda()
        free = order[ns + int(have.sum()):]
        # (a list as long as the pool, which is the same for every seed)
        s["free"] = torch.zeros(max(pages, B * case["max_pages"] // 2 + case["max_pages"] + ns + 8), dtype=torch.int32,
                                device="cuda")
        s["free"][:len(free)] = free.int().cuda()
        s["n_free"] = torch.tensor([len(free)], dtype=torch.int32, device="cuda")
        s["past"], s["table"] = past.int().cuda(), table.int().cuda()
    return s


def _attn_plain(s):
    c = s["case"]
    B, Hq, Hkv, D, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G, n = Hq // Hkv, c["prefix_pages"] * P
    lens = s["lens"].long()
    first = torch.where(lens >= n, n, 0) if s["shares"] is None else torch.where(s["shares"] & (lens >= n), n, 0)
    q = s["q"].float().view(B, Hkv, G, D)
    kp = s["k"][s["shared"].long()].flatten(0, 1).float() * s["k_scale"]
    vp = s["v"][s["shared"].long()].flatten(0, 1).float() * s["v_scale"]
    rows = q.transpose(0, 1).reshape(Hkv, B * G, D)
    sp = torch.matmul(rows, kp.permute(1, 2, 0)) * s["scale"]
    sp = sp.view(Hkv, B, G, n).masked_fill((first == 0)[None, :, None, None], -math.inf)
    j = first[:, None] + torch.arange(c["max_own"], device="cuda")[None, :]
    seen = j < lens[:, None]
    at = torch.where(seen, j, 0)
    page = torch.gather(s["table"].long(), 1, at // P)
    ko = s["k"][page, at % P].float() * s["k_scale"]
    vo = s["v"][page, at % P].float() * s["v_scale"] * seen[:, :, None, None]
    so = torch.matmul(q, ko.permute(0, 2, 3, 1)) * s["scale"]
    so = so.masked_fill(~seen[:, None, None, :], -math.inf).transpose(0, 1)
    m = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    sp, so = torch.exp(sp - m), torch.exp(so - m)
    l = sp.sum(-1, keepdim=True) + so.sum(-1, keepdim=True)
    o = torch.matmul(sp.view(Hkv, B * G, n), vp.transpose(0, 1)).view(Hkv, B, G, D)
    o = o + torch.matmul(so.transpose(0, 1), vo.transpose(1, 2)).transpose(0, 1)
    o = o / torch.where(l > 0, l, torch.ones_like(l))
    back = lambda t: t.transpose(0, 1).reshape(B, Hq, -1)  # noqa: E731
    return back(o).to(s["q"].dtype), back(m + torch.log(l))[..., 0]


def _router_plain(s):
    c = s["case"]
    T, E, k, n = c["T"], c["E"], c["k"], c["groups"]
    x = s["logits"].double()  # (which of two scores is larger has to be right)
    if c["score"] == "softmax":
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    key = p if s["bias"] is None else p + s["bias"].double()
    if s["bias"] is None:
        key = x  # the order of the scores without their rounding
    if c["top_groups"] < n:
        a = (p if s["bias"] is None else key).view(T, n, E // n)
        top = torch.sort(a, dim=-1, descending=True)[0]
        score = top[..., 0] + top[..., 1] if c["group_score"] == "top2" else top[..., 0]
        best = torch.sort(score, dim=-1, descending=True, stable=True)[1][:, :c["top_groups"]]
        keep = torch.zeros(T, n, dtype=torch.bool, device="cuda").scatter_(1, best, True)
        key = key.view(T, n, E // n).masked_fill(~keep[:, :, None], -math.inf).view(T, E)
    ids = torch.sort(key, dim=-1, descending=True, stable=True)[1][:, :k]
    w = torch.gather(p, 1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.int(), (w * c["scale"]).float()


def _plan_plain(s):
    c = s["case"]
    B, P, T, ns = c["B"], c["page"], _tokens(c), c["shared"]
    past, new, free = s["past"].long(), s["new"].long(), s["n_free"].long()
    have = (past + P - 1) // P
    need = (past + new + P - 1) // P - have
    fits = ((torch.cumsum(need, 0) <= free) | (need == 0)) & (torch.cumsum(new, 0) <= T)
    fits &= past + new <= c["max_pages"] * P
    new, need = torch.where(fits, new, 0), torch.where(fits, need, 0)
    starts = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    starts[1:] = torch.cumsum(new, 0)
    taken = torch.cumsum(need, 0) - need
    # the pages of the rows
    at = torch.arange(c["max_pages"], device="cuda")[None, :]
    fresh = (at >= have[:, None]) & (at < (have + need)[:, None])
    which = (free - 1 - taken[:, None] - (at - have[:, None])).clamp(0, s["free"].shape[0] - 1)
    table = torch.where(fresh, s["free"][which], s["table"])
    if ns:
        first = s["shares"] & (past == ns * P) & (new > 0)
        n0 = min(ns, c["max_pages"])
        table[:, :n0] = torch.where(first[:, None], s["shared"][None, :n0], table[:, :n0])
    s["table"].copy_(table)
    # the tokens
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(starts[1:], t, right=True)
    there = b < B
    b = b.clamp(max=B - 1)
    pos = past[b] + t - starts[b]
    page = table[b, (pos // P).clamp(0, c["max_pages"] - 1)].long()
    slots = torch.where(there, page * P + pos % P, -1)
    return (torch.where(there, pos, 0).int(), slots, torch.where(there, b, -1).int(), starts.int(), (past + new).int(),
            (free - need.sum()).int(), s["table"])


def _release_plain(s):
    c = s["case"]
    P = c["page"]
    past, free = s["past"].long(), s["n_free"].long()
    at = torch.arange(c["max_pages"], device="cuda")[None, :]
    skip = torch.where(s["shares"], c["shared"], 0)
    goes = s["ended"][:, None] & (at >= skip[:, None]) & (at < ((past + P - 1) // P)[:, None])
    place = free + torch.cumsum(goes.view(-1), 0) - 1
    n = s["free"].shape[0]
    out = torch.cat((s["free"], s["free"][:1]))  # the last place takes what does not go
    out[torch.where(goes.view(-1), place, n)] = s["table"].view(-1)
    s["free"].copy_(out[:n])
    return s["free"], (free + goes.sum()).int(), torch.where(s["ended"], 0, past).int()


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"attn": _attn_plain, "router": _router_plain, "plan": _plan_plain, "release": _release_plain}[c["op"]](s)
    import mixture_experts_decode_gb300 as moe
    if c["op"] == "attn":
        return moe.shared_prefix_attention(s["q"], s["k"], s["v"], s["shared"], c["prefix_pages"] * c["page"], s["table"],
                                           s["lens"], shares=s["shares"], scale=s["scale"], k_scale=s["k_scale"],
                                           v_scale=s["v_scale"], workspace=s["ws"], return_lse=True)
    if c["op"] == "router":
        return moe.router_grouped_topk(s["logits"], c["k"], bias=s["bias"], score=c["score"], groups=c["groups"],
                                       top_groups=c["top_groups"], group_score=c["group_score"],
                                       renormalize=c["renorm"], scale=c["scale"])
    shared = s["shared"] if c["shared"] else None
    if c["op"] == "plan":
        p = moe.plan_pages(s["past"], s["new"], s["table"], s["free"], s["n_free"], c["page"], _tokens(c),
                           shared_pages=shared, shares=s["shares"])
        return p.positions, p.slots, p.seq_ids, p.starts, p.seq_lens, p.n_free, s["table"]
    lens, n_free = moe.release_pages(s["table"], s["past"], s["ended"], s["free"], s["n_free"], c["page"],
                                     shared=c["shared"], shares=s["shares"])
    return s["free"], n_free, lens


def work(case):
    if case["op"] == "attn":
        B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
        sharing = B - len(range(3, B, 5)) if case["others"] else B
        prefix, mine = case["prefix_pages"] * case["page"], B * case["max_own"] / 3
        return {"bytes": 2 * (prefix + mine) * Hkv * D * SIZES[case["cache"]] + 4 * B * Hq * D + 4 * B * Hq,
                "flops": 4 * (sharing * prefix + mine) * Hq * D}
    if case["op"] == "router":
        T, E = case["T"], case["E"]
        return {"bytes": T * E * SIZES[case["dtype"]] + (4 * E if case["bias"] else 0) + 8 * T * case["k"],
                "flops": T * E * (8 + case["k"])}
    B, P = case["B"], case["page"]
    mean = case["max_past"] / max(1.0, math.log(case["max_past"]))
    if case["op"] == "plan":
        T = _tokens(case)
        return {"bytes": 16 * T + 8 * T // P + 16 * B + 4 * min(B, T) + 4 * B * case["shared"] * case["begin"],
                "flops": 8 * T + 16 * B}
    return {"bytes": 8 * B * case["ends"] * mean / P + 13 * B, "flops": B * case["ends"] * mean / P + 8 * B}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        B, Hq, Hkv, D, P = case["B"], case["Hq"], case["Hkv"], case["D"], case["page"]
        out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
        G = Hq // Hkv
        # the same keys and values in 64 bits for all that read them, one head after the other
        shared = s["shared"].tolist()
        tables, lens = s["table"].tolist(), s["lens"].tolist()
        sharing = [True] * B if s["shares"] is None else s["shares"].tolist()
        for h in range(Hkv):
            kp = torch.cat([s["k"][p, :, h] for p in shared]).double() * s["k_scale"]
            vp = torch.cat([s["v"][p, :, h] for p in shared]).double() * s["v_scale"]
            for b in range(B):
                if not lens[b]:
                    continue
                first = len(shared) if sharing[b] and lens[b] >= len(shared) * P else 0
                last = -(-lens[b] // P)
                mine = torch.tensor(tables[b][first:last], dtype=torch.int64, device="cuda")
                n = lens[b] - first * P
                k = s["k"][mine, :, h].reshape(-1, D)[:n].double() * s["k_scale"]
                v = s["v"][mine, :, h].reshape(-1, D)[:n].double() * s["v_scale"]
                if first:
                    k, v = torch.cat((kp, k)), torch.cat((vp, v))
                heads = slice(h * G, (h + 1) * G)
                score = s["q"][b, heads].double() @ k.T * s["scale"]
                lse[b, heads] = torch.logsumexp(score, -1)
                out[b, heads] = torch.softmax(score, -1) @ v
        return out, lse
    if case["op"] == "router":
        import numpy as np
        x = s["logits"].double().cpu().numpy()
        T, E = x.shape
        size = E // case["groups"]
        score = (torch.softmax if case["score"] == "softmax" else lambda a, _: torch.sigmoid(a))(s["logits"].double(), -1)
        score = score.cpu().numpy()
        key = x if s["bias"] is None else score + s["bias"].double().cpu().numpy()
        live = np.ones((T, E), dtype=bool)
        if case["top_groups"] < case["groups"]:
            by = (score if s["bias"] is None else key).reshape(T, case["groups"], size)
            part = np.partition(by, size - 2, -1)[..., -2:]
            worth = part.sum(-1) if case["group_score"] == "top2" else part[..., 1]
            order = np.argsort(-worth, axis=-1, kind="stable")[:, :case["top_groups"]]
            chosen = np.zeros(worth.shape, dtype=bool)
            np.put_along_axis(chosen, order, True, -1)
            live = np.repeat(chosen, size, axis=1)
        rank = np.where(live, key, -np.inf)
        ids = np.empty((T, case["k"]), dtype=np.int64)
        for j in range(case["k"]):  # (argmax takes the first of equal ones)
            ids[:, j] = rank.argmax(-1)
            np.put_along_axis(rank, ids[:, j:j + 1], -np.inf, -1)
        w = np.take_along_axis(score, ids, -1)
        if case["renorm"]:
            w = w / w.sum(-1, keepdims=True)
        return torch.from_numpy(ids).int().cuda(), torch.from_numpy(w * case["scale"]).cuda()
    P, past, table = case["page"], s["past"].tolist(), s["table"].cpu().clone()
    shares, free, n = s["shares"].tolist(), s["free"].cpu().clone(), int(s["n_free"])
    if case["op"] == "release":
        lens = list(past)
        for b, ended in enumerate(s["ended"].tolist()):
            if ended:
                row = table[b, case["shared"] if shares[b] else 0:-(-past[b] // P)]
                free[n:n + len(row)] = row
                n, lens[b] = n + len(row), 0
        return free.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    T, new = _tokens(case), s["new"].tolist()
    pos, slots, seqs = torch.zeros(T, dtype=torch.int32), torch.full((T,), -1), torch.full((T,), -1, dtype=torch.int32)
    starts, lens, wanted, asked, t, top = [0], [], 0, 0, 0, n
    for b in range(case["B"]):
        end = past[b] + new[b]
        need = -(-end // P) - -(-past[b] // P)
        wanted, asked = wanted + need, asked + new[b]
        if (need == 0 or wanted <= top) and asked <= T and end <= case["max_pages"] * P:
            if shares[b] and new[b] and case["shared"] and past[b] == case["shared"] * P:
                table[b, :case["shared"]] = s["shared"].cpu()[:case["max_pages"]]
            for i in range(-(-past[b] // P), -(-end // P)):
                n -= 1
                table[b, i] = free[n]
            p = torch.arange(past[b], end)
            pos[t:t + new[b]], seqs[t:t + new[b]] = p.int(), b
            slots[t:t + new[b]] = table[b, p // P].long() * P + p % P
            t += new[b]
            lens.append(end)
        else:
            lens.append(past[b])
        starts.append(t)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    return pos.cuda(), slots.cuda(), seqs.cuda(), i32(starts), i32(lens), i32([n]), table.cuda()
