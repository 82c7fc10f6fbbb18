"""Plain 64-bit and integer references of the serving step's operators (not collected by pytest)."""
from __future__ import annotations

import numpy as np
import torch


def router(logits, k, bias, score, groups, top_groups, group_score, renorm, scale):
    """(ids, weights) by the definition, in float64 on the host; absent: -1 and 0."""
    x = logits.double().cpu().numpy()
    T, E = x.shape
    x = np.where(np.isnan(x), -np.inf, x)
    with np.errstate(all="ignore"):
        if score == "softmax":
            p = np.exp(x - x.max(-1, keepdims=True))
            p = p / p.sum(-1, keepdims=True)
        else:
            p = np.where(x > 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
        b = np.zeros(E) if bias is None else bias.double().cpu().numpy()
        flat = bool((b == b[0]).all()) and np.isfinite(b[0])
        key = x.copy() if flat else p + b  # (one bias for all: the logits' own order)
        key[(x == -np.inf) | np.isnan(key)] = -np.inf
    size = E // groups
    live = np.ones((T, E), dtype=bool)
    if top_groups < groups:
        by = (p + b if flat and group_score == "top2" else key).copy()
        by[key == -np.inf] = -np.inf
        by = np.sort(by.reshape(T, groups, size), -1)
        with np.errstate(all="ignore"):
            worth = by[..., -1] + by[..., -2] if group_score == "top2" else by[..., -1]
        worth = np.where(np.isnan(worth), -np.inf, worth)
        chosen = np.zeros((T, groups), dtype=bool)
        np.put_along_axis(chosen, np.argsort(-worth, axis=-1, kind="stable")[:, :top_groups], True, -1)
        live = np.repeat(chosen, size, axis=1)
    row = np.where(live, key, -np.inf)
    ids = np.argsort(-row, axis=-1, kind="stable")[:, :k]
    there = np.take_along_axis(row, ids, -1) > -np.inf
    v, xs = np.take_along_axis(p, ids, -1), np.take_along_axis(x, ids, -1)
    if renorm:
        if score == "sigmoid":   # the ratios of scores that are all tiny are those of their exponentials
            tiny = np.where(there, v, 0).sum(-1) < 1e-200
            top = np.max(np.where(there, xs, -np.inf), -1, keepdims=True, initial=-1e300)
            with np.errstate(all="ignore"):
                v = np.where(tiny[:, None], np.exp(xs - top), v)
        with np.errstate(all="ignore"):
            v = v / np.where(there, v, 0).sum(-1, keepdims=True)
    return np.where(there, ids, -1), np.where(there, v * scale, 0.0)


def plan(past, new, table, free, n_free, page, T, shared=(), shares=None):
    """moe_plan_pages request by request on lists: (positions, slots, seq_ids, starts, lens, n_free, table, refused)."""
    table = [list(r) for r in table]
    most = len(table[0]) if table else 0
    pos, slots, seqs, starts, lens = [0] * T, [-1] * T, [-1] * T, [0], []
    t, left, wanted, asked, refused = 0, n_free, 0, 0, False
    for b, (p, n) in enumerate(zip(past, new)):
        ok = p >= 0 and n >= 0
        if ok:
            need = -(-(p + n) // page) - -(-p // page)
            wanted, asked = wanted + need, asked + n
            ok = asked <= T and (need == 0 or wanted <= n_free) and p + n <= min(most * page, 2 ** 31 - 1)
            refused |= not ok and n > 0
        else:
            refused = True
        if ok:
            if shared and n and p == len(shared) * page and (shares is None or shares[b]):
                table[b][:len(shared)] = shared[:most]
            for i in range(-(-p // page), -(-(p + n) // page)):
                left -= 1
                table[b][i] = free[left]
            for j in range(p, p + n):
                pos[t], seqs[t], slots[t] = j, b, table[b][j // page] * page + j % page
                t += 1
        lens.append(p + n if ok else p)
        starts.append(t)
    return pos, slots, seqs, starts, lens, left, table, refused


def release(table, lens, ended, free, n_free, page, shared=0, shares=None):
    """moe_release_pages on lists: (free, n_free, lens)."""
    free, lens = list(free), list(lens)
    for b, e in enumerate(ended):
        if e:
            row = table[b][:-(-max(lens[b], 0) // page)][shared if shares is None or shares[b] else 0:]
            for pg in row:
                if n_free < len(free):
                    free[n_free] = pg
                    n_free += 1
            lens[b] = 0
    return free, n_free, lens


def random_plan(g, B, page, most, past_max, new_max, room=1.0, ns=0):
    """Host lists of a random state: past, new, table, free, n_free, shared, shares."""
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    shares = [r(0, 3) > 0 for _ in range(B)]
    past, new = [], []
    for b in range(B):
        fresh = r(0, 2) == 0
        past.append((ns * page if shares[b] else 0) if fresh else r(0, past_max))
        new.append(r(0, new_max))
    have = [-(-p // page) for p in past]
    need = sum(-(-(p + n) // page) - h for p, n, h in zip(past, new, have))
    pages = torch.randperm(sum(have) + ns + need + 5, generator=g).tolist()
    table = [[-1] * most for _ in range(B)]
    shared = [pages.pop() for _ in range(ns)]
    for b in range(B):
        for i in range(min(have[b], most)):
            table[b][i] = pages.pop()
    n_free = min(len(pages), int(need * room))
    return past, new, table, pages, n_free, shared, shares
