"""moe_shared_prefix_attention against attention over whole sequences in 64 bits.

Bounds as derived in _block_refs.attention.  With an E4M3 cache and a BF16 query
the weights of the prefix are one FP16 value each, 2^-11 of themselves: that
share of sum p|v| comes on top."""
import math

import pytest
import torch

import mixture_experts_decode_gb300 as moe
import _block_refs as refs

pytestmark = pytest.mark.gpu
BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def make(dev, B, Hq, Hkv, D, page, prefix, own, dtype=BF, cache=None, seed=0, others=(), order="nhd", q_std=1.5, spare=3):
    """own: tokens behind the prefix of each sequence (a number or a list); others: the sequences that do not share (own
    tokens alone).  A prefix that ends inside a page has its last rows copied into the sequences' own pages."""
    g = torch.Generator(device=dev).manual_seed(seed)
    cache = cache or dtype
    own = [own] * B if isinstance(own, int) else list(own)
    ns, cut = -(-prefix // page), prefix % page
    lens = [n if b in others else prefix + n for b, n in enumerate(own)]
    used = [-(-n // page) for n in lens]
    mine = [u - (0 if b in others else prefix // page) for b, u in enumerate(used)]
    pages = ns + sum(max(m, 0) for m in mine) + spare
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    shared = [perm.pop() for _ in range(ns)]
    table = torch.full((B, max(used + [ns, 1])), -7, dtype=torch.int32)
    shape = (pages, page, Hkv, D) if order == "nhd" else (pages, Hkv, page, D)
    ks, vs = (0.03, 0.02) if cache == E4 else (1.0, 1.0)
    rnd = lambda sc: (torch.randn(shape, generator=g, device=dev) / sc).to(cache)  # noqa: E731
    k, v = rnd(ks), rnd(vs)
    if order == "hnd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    for b in range(B):
        first = 0 if b in others else prefix // page
        table[b, :first] = torch.tensor(shared[:first], dtype=torch.int32)
        for i in range(first, used[b]):
            table[b, i] = perm.pop()
        if b not in others and cut and used[b] > first:
            for t in (k, v):
                raw = t.view(torch.uint8) if cache == E4 else t
                raw[int(table[b, first]), :cut] = raw[shared[first], :cut]
    q = (torch.randn(B, Hq, D, generator=g, device=dev) * q_std).to(dtype)
    shares = None
    if others:
        shares = torch.tensor([b not in others for b in range(B)], device=dev)
    return dict(q=q, k=k, v=v, table=table.to(dev), lens=torch.tensor(lens, dtype=torch.int32, device=dev), ks=ks, vs=vs,
                shared=torch.tensor(shared, dtype=torch.int32, device=dev), prefix=prefix, shares=shares)


def call(c, scale=None, ws=None, **kw):
    return moe.shared_prefix_attention(c["q"], c["k"], c["v"], c["shared"], c["prefix"], c["table"], c["lens"], c["shares"],
                                       scale=scale, k_scale=c["ks"], v_scale=c["vs"], workspace=ws, return_lse=True, **kw)


def check(c, scale=None, ws=None, what=""):
    q = c["q"]
    out, lse = call(c, scale, ws)
    torch.cuda.synchronize()
    s = q.shape[2] ** -0.5 if scale is None else scale
    ro, rl, ob, lb = refs.attention(q, c["k"], c["v"], c["table"], c["lens"], s, 0, 0, c["ks"], c["vs"])
    if c["k"].dtype == E4 and q.dtype == BF:
        ab = refs.attention(q, c["k"], c["v"].double().abs(), c["table"], c["lens"], s, 0, 0, c["ks"], c["vs"])[0]
        ob = ob + 2.0 ** -11 * ab
    assert out.dtype == q.dtype and not torch.isnan(out).any(), what
    err = (out.double() - ro).abs() - ob
    assert err.max() <= 0, f"{what}: out beyond its bound by {err.max().item():.3g} at {torch.nonzero(err > 0)[:4].tolist()}"
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty), what
    e = ((lse.double() - rl).abs() - lb)[~empty]
    assert e.numel() == 0 or e.max() <= 0, f"{what}: lse beyond its bound by {e.max().item():.3g}"
    return out, lse


def enough(Hkv, D, prefix, cache):
    """Sequences from which the prefix is read by itself (below, each reads its own row)."""
    return max(3 if cache == E4 else 2, math.ceil((64e6 if cache == E4 else 12e6) / (2 * prefix * Hkv * D)) + 1)


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 144, 192, 256])
def test_head_sizes(cuda_device, D, dtype, cache):
    prefix = 24 * 130
    B = enough(3, D, prefix, cache)
    check(make(cuda_device, B, 6, 3, D, 24, prefix, [(i * 7) % 40 for i in range(B)], dtype, cache, seed=D, others=(1,)),
          what=f"D={D}")


@pytest.mark.parametrize("prefix", [1, 64, 511, 512, 513, 575, 576, 577, 639, 640, 641, 777, 1151, 1152, 3001])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, E4)])
def test_prefix_lengths(cuda_device, prefix, dtype, cache):
    B = min(enough(4, 128, prefix, cache), 130)
    check(make(cuda_device, B, 8, 4, 128, 16, prefix, [(i * 11) % 50 for i in range(B)], dtype, cache, seed=prefix),
          what=f"prefix={prefix}")


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 1), (9, 3), (20, 1), (40, 8), (64, 4), (128, 1)])
@pytest.mark.parametrize("B", [2, 13, 40])
def test_rows_of_a_head(cuda_device, Hq, Hkv, B):
    """2 to 5120 rows a key-value head: parts of a tile, one tile, two, and several groups of them."""
    prefix = max(512, math.ceil(12e6 / (2 * (B - 1) * Hkv * 64)))
    own = [(i * 7) % 20 for i in range(B)]
    check(make(cuda_device, B, Hq, Hkv, 64, 16, prefix, own, HF, seed=Hq + B, others=(1,) if B > 2 else ()), what=f"{Hq}/{Hkv} B={B}")


@pytest.mark.parametrize("D,cache", [(128, BF), (256, BF), (128, E4), (256, E4)])
def test_many_rows_of_wide_heads(cuda_device, D, cache):
    prefix = 8200 if cache == E4 else 4100
    check(make(cuda_device, 33, 16, 1, D, 32, prefix, [i % 9 for i in range(33)], BF, cache, seed=D), what=f"D={D}")


@pytest.mark.parametrize("D,prefix,dtype,cache", [(64, 16000, HF, HF), (64, 16001, BF, E4), (128, 9000, BF, BF), (128, 9000, BF, E4),
                                                  (256, 4000, HF, HF), (256, 4000, BF, E4)])
@pytest.mark.parametrize("G", [1, 6])
def test_many_tiles_a_block(cuda_device, D, prefix, dtype, cache, G):
    """A dozen key tiles and more for each block, and calls behind one another: the same bits every time."""
    c = make(cuda_device, 50, 16 * G, 16, D, 32, prefix, [(i * 7) % 60 for i in range(50)], dtype, cache, seed=D + G)
    want, wl = check(c, what=f"D={D}")
    ws = moe.shared_prefix_workspace(50, 16 * G, 16, D)
    outs = [call(c, ws=ws) for _ in range(20)]
    torch.cuda.synchronize()
    assert moe.device_error(cuda_device) == 0
    assert all(torch.equal(o, want) and torch.equal(s, wl) for o, s in outs)


@pytest.mark.parametrize("page", [1, 3, 8, 13, 100, 256])
def test_page_sizes(cuda_device, page):
    B = enough(2, 128, 999, BF)
    check(make(cuda_device, B, 4, 2, 128, page, 999, [(i * 37) % 100 for i in range(B)], BF, seed=page), what=f"page={page}")


@pytest.mark.parametrize("cache", [BF, E4])
def test_long_prefix(cuda_device, cache):
    prefix = 70000 if cache == E4 else 40000
    check(make(cuda_device, 3, 16, 2, 128, 64, prefix, [5, 0, 300], BF, cache, seed=7, q_std=3.0), what="long")
    if cache == BF:   # small pages: more of them than a block holds the places of
        check(make(cuda_device, 2, 16, 1, 128, 1, 50000, [5, 9], BF, cache, seed=7), what="pages of one")


def test_growing_scores(cuda_device):
    """Keys that grow along the prefix move the reference of the exponents again and again; shrinking ones leave a long tail."""
    for dtype, cache in ((BF, BF), (HF, HF), (BF, E4)):
        B = enough(1, 128, 4096, cache)
        for rising in (True, False):
            c = make(cuda_device, B, 4, 1, 128, 32, 4096, [(i * 5) % 41 for i in range(B)], dtype, cache, seed=3)
            flat = (c["k"].double() * c["ks"])
            for i, pg in enumerate(c["shared"].tolist()):
                x = (i if rising else 127 - i) / 16
                flat[pg] = flat[pg] * 0.05 + x * c["q"][0, 0].double() / c["q"][0, 0].double().norm()
            c["k"] = (flat / c["ks"]).to(c["k"].dtype)
            check(c, scale=1.0, what=f"rising={rising}")


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-3, 2.0])
@pytest.mark.parametrize("cache", [HF, E4])
def test_scales(cuda_device, scale, cache):
    B = enough(2, 64, 1300, cache)
    check(make(cuda_device, B, 8, 2, 64, 16, 1300, [(i * 3) % 21 for i in range(B)], HF, cache, seed=5), scale=scale,
          what=f"scale={scale}")


def test_sequences_that_end_inside_the_prefix_or_are_empty(cuda_device):
    c = make(cuda_device, 6, 8, 2, 128, 16, 5000, [0, 10, 20, 30, 0, 5], BF, seed=11, others=(4,))
    c["lens"] = torch.tensor([4999, 0, 5020, 37, 0, 5000], dtype=torch.int32, device=cuda_device)
    c["table"][5, 313:] = 1 << 29       # never looked up
    out, lse = check(c)
    assert bool((out[1] == 0).all()) and bool((out[4] == 0).all()) and bool((lse[1] == -math.inf).all())


@pytest.mark.parametrize("order", ["nhd", "hnd"])
def test_strides(cuda_device, order):
    c = make(cuda_device, 5, 8, 2, 128, 16, 6333, [5, 0, 17, 40, 2], BF, seed=12, order=order)
    want, _ = check(c)
    g = torch.zeros(5, 3, 8, 136, dtype=BF, device=cuda_device)
    g[:, 1, :, :128] = c["q"]
    c["q"] = g[:, 1, :, :128]
    wide = torch.full((5, c["table"].shape[1] + 5), -9, dtype=torch.int32, device=cuda_device)
    wide[:, :-5] = c["table"]
    c["table"] = wide[:, :-5]
    out, _ = check(c)
    assert torch.equal(out, want)
    buf = torch.full((5 * 8 * 128 + 5,), 7.0, dtype=BF, device=cuda_device)
    got, _ = call(c, out=buf[1:-4].view(5, 8, 128))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and buf[0] == 7 and bool((buf[-4:] == 7).all())


def test_masked_places_are_not_read(cuda_device):
    """Infinities and NaN behind the prefix's end, in rows that a sequence does not see, and in the prefix for those that do
    not share it."""
    c = make(cuda_device, 4, 8, 2, 128, 16, 8008, [10, 0, 33, 17], BF, seed=13, others=(2,))
    want, wl = check(c)
    last = int(c["shared"][-1])
    c["k"][last, 8:] = float("nan")
    c["v"][last, 8:] = float("inf")
    out, lse = call(c)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    c["v"][int(c["shared"][0]), 3] = float("nan")
    c["k"][int(c["shared"][0]), 3] = float("inf")
    out, lse = call(c)
    torch.cuda.synchronize()
    assert torch.equal(out[2], want[2]) and torch.equal(lse[2], wl[2])
    assert bool(torch.isnan(out[[0, 1, 3]]).all())


def test_infinities_and_nan_among_visible_values(cuda_device):
    """Wherever in the prefix they lie, however small their key's weight: the dim is not finite, the others are as they were."""
    for dtype, cache in ((BF, BF), (HF, HF), (BF, E4)):
        c = make(cuda_device, 17, 8, 2, 128, 16, 8192, [10 + i for i in range(17)], dtype, cache, seed=23, others=(2,), q_std=6.0)
        want, _ = check(c)
        for i, (pg, row) in enumerate(((0, 0), (100, 7), (511, 15))):
            v = c["v"].clone()
            v[int(c["shared"][pg]), row, 1, 5 + i] = float("nan") if cache == E4 or i == 1 else float("-inf")
            out, _ = call(dict(c, v=v))
            torch.cuda.synchronize()
            bad = ~torch.isfinite(out)
            seen = torch.zeros_like(bad)
            seen[:, 4:, 5 + i] = True
            seen[2] = False
            assert torch.equal(bad, seen) and torch.equal(out[~bad], want[~bad])


def test_infinite_keys(cuda_device):
    """A score of -inf leaves its key out, one of +inf makes its head's output NaN, in the shared part too."""
    for dtype in (BF, HF):
        for pg, row in ((0, 0), (100, 7), (511, 15)):
            c = make(cuda_device, 17, 8, 2, 128, 16, 8192, [10 + i for i in range(17)], dtype, seed=29, others=(2,))
            sign = torch.where(torch.rand(17, 4, device=cuda_device) < 0.5, -1.0, 1.0).to(dtype)
            c["q"][:, 4:, 9] = sign
            k = c["k"].clone()
            c["k"][int(c["shared"][pg]), row, 1, 9] = 6e4    # (weight 0 where the query's value is -1)
            want, _ = call(c)
            k[int(c["shared"][pg]), row, 1, 9] = float("inf")
            out, _ = call(dict(c, k=k))
            torch.cuda.synchronize()
            nan = torch.zeros_like(out, dtype=torch.bool)
            nan[:, 4:] = (sign > 0)[..., None]
            nan[2] = False
            assert torch.equal(torch.isnan(out), nan) and torch.equal(out[~nan], want[~nan])


@pytest.mark.parametrize("cache", [BF, E4])
def test_caches_whose_offsets_pass_32_bits(cuda_device, cache):
    B = enough(2, 128, 640, cache)
    c = make(cuda_device, B, 8, 2, 128, 64, 640, [(i * 5) % 64 for i in range(B)], BF, cache, seed=37)
    want, wl = check(c)
    pages = c["k"].shape[0]
    step = -(-(2 ** 32 + 2 ** 28) // pages) // 16 * 16 + 16     # elements: the last pages begin behind 2^32
    buf = torch.empty(2 * pages * step, dtype=torch.uint8 if cache == E4 else cache, device=cuda_device)
    far = []
    for i, t in enumerate((c["k"], c["v"])):
        f = buf.as_strided(t.shape, (step, *t.stride()[1:]), i * pages * step)
        f.copy_(t.view(torch.uint8) if cache == E4 else t)
        far.append(f.view(E4) if cache == E4 else f)
    out, lse = call(dict(c, k=far[0], v=far[1]))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_out_may_be_the_query(cuda_device):
    for prefix in (100, 8000):
        c = make(cuda_device, 9, 8, 2, 128, 16, prefix, [3 * i for i in range(9)], BF, seed=31)
        want, wl = check(c)
        out, lse = call(c, out=c["q"])
        torch.cuda.synchronize()
        assert out.data_ptr() == c["q"].data_ptr() and torch.equal(out, want) and torch.equal(lse, wl)


def test_a_page_outside_the_cache_is_left_out(cuda_device):
    c = make(cuda_device, 4, 8, 2, 128, 16, 8000, [10, 0, 33, 17], BF, seed=14)
    for bad in (-1, 1 << 30, c["k"].shape[0]):
        c["shared"][5] = bad
        c["table"][:, 5] = bad
        check(c)
        assert moe.device_error(cuda_device) == 0x8


def test_nothing_shared_is_paged_attention(cuda_device):
    c = make(cuda_device, 4, 8, 2, 64, 16, 0, [10, 0, 33, 170], BF, seed=15)
    out, lse = check(c)
    want, wl = moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    for prefix in (64, 8192):
        c = make(cuda_device, 4, 8, 2, 128, 16, prefix, [10, 0, 33, 170], BF, seed=15)
        c["shares"] = torch.zeros(4, dtype=torch.uint8, device=cuda_device)
        check(c)


def test_a_kept_workspace_serves_both_calls(cuda_device):
    ws = moe.shared_prefix_workspace(64, 16, 2, 128, cuda_device)
    for i, (B, prefix) in enumerate(((64, 700), (3, 15000), (1, 64), (40, 129), (33, 1000), (2, 25000))):
        c = make(cuda_device, B, 16, 2, 128, 16, prefix, [(j * 37) % 400 for j in range(B)], BF, seed=i)
        out, lse = check(c, ws=ws)
        again, l2 = call(c, ws=ws)
        assert torch.equal(out, again) and torch.equal(lse, l2)
        a = moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], workspace=ws)
        b = moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"])
        assert torch.equal(a, b)
    assert int(ws[:4096].sum()) == 0


def test_two_streams_and_two_graphs(cuda_device):
    cs = [make(cuda_device, 20, 16, 2, 128, 16, 3000, [(j * 37) % 400 for j in range(20)], BF, seed=i) for i in (1, 2)]
    want = [call(c) for c in cs]
    wss = [moe.shared_prefix_workspace(20, 16, 2, 128, cuda_device) for _ in cs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in cs]
    for c, ws in zip(cs, wss):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(c, ws=ws))
        graphs.append(g)
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)


def test_lengths_move_under_a_captured_call(cuda_device):
    c = make(cuda_device, 6, 8, 2, 128, 16, 4800, [100] * 6, BF, seed=21)
    ws = moe.shared_prefix_workspace(6, 8, 2, 128, cuda_device)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = call(c, ws=ws)
    for lens in ([4800, 4801, 4880, 4900, 0, 100], [4799, 4900, 4810, 4820, 4830, 4840]):
        c["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want, wl = check(c)
        assert torch.equal(out, want) and torch.equal(lse, wl)


def test_outputs_over_the_query(cuda_device):
    c = make(cuda_device, 5, 8, 2, 128, 16, 6333, [5, 0, 17, 40, 2], BF, seed=22)
    want, _ = check(c)
    got, _ = call(c, out=c["q"])
    torch.cuda.synchronize()
    assert torch.equal(got, want)
