"""GPU parity of moe_rope_append, moe_norm_residual and moe_matvec4 against
plain implementations in 64 bits, with bounds derived in _block_refs."""
import math

import pytest
import torch

import _block_refs as refs
import mixture_experts_decode_gb300 as moe

pytestmark = pytest.mark.gpu
BF, HF, E4, F32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float32


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0


def within(got, want, bound, dtype, what):
    """|got - want| <= the type's half step of the value (or of its smallest normal) + bound."""
    tiny = torch.finfo(dtype).tiny * refs.half_step(dtype) * 2
    tol = refs.half_step(dtype) * (want.abs() + bound) + bound + tiny
    err = (got.double() - want).abs() - tol
    assert not torch.isnan(got.float()).any(), what
    assert err.numel() == 0 or err.max() <= 0, f"{what}: beyond its bound by {err.max().item():.3g}"


# ------------------------------------------------------------------ rotary ---

def rope_case(dev, T, Hq, Hkv, D, rot, page=16, dtype=BF, cache=None, seed=0, max_pos=5000, scaling="none"):
    g = torch.Generator(device=dev).manual_seed(seed)
    cache = cache or dtype
    pages = T // page + 3
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    qkv = rnd(T, Hq + 2 * Hkv, D).to(dtype)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    c = dict(q=q, k=k, v=v, kc=rnd(pages, page, Hkv, D).to(cache), vc=rnd(pages, page, Hkv, D).to(cache),
             pos=torch.randint(0, max_pos, (T,), generator=g, device=dev, dtype=torch.int32),
             slots=torch.randperm(pages * page, generator=g, device=dev)[:T].contiguous(),
             freqs=moe.rope_freqs(rot, scaling=scaling, factor=4.0, device=dev) if rot else
             torch.empty(0, dtype=torch.float64, device=dev), rot=rot, ks=0.05 if cache == E4 else 1.0,
             vs=0.02 if cache == E4 else 1.0)
    return c


def raw(t):
    return t.contiguous().view(torch.uint8 if t.dtype == E4 else torch.int16)


def rope_check(c, interleaved=False, mscale=1.0, what="", q_out=None):
    before = raw(c["kc"]).clone(), raw(c["vc"]).clone()
    q_in, k_in, v_in = c["q"].clone(), c["k"].clone(), c["v"].clone()
    got = moe.rope_append(c["q"], c["k"], c["v"], c["pos"], c["slots"], c["freqs"], c["kc"], c["vc"],
                          interleaved=interleaved, mscale=mscale, k_scale=c["ks"], v_scale=c["vs"], q_out=q_out)
    torch.cuda.synchronize()
    # the terms' size times four FP32 half steps: sine, product, sum; the
    # angle's fraction is off by 2^-24 of itself (pi at most) and 2^-32 turns
    rel = 8 * refs.U32 + 2.0 ** -22
    want, size = refs.rotate(q_in, c["pos"], c["freqs"], c["rot"], interleaved, mscale)
    within(got, want, size * rel, got.dtype, what + " q")
    slots = c["slots"]
    P, cache = c["kc"].shape[1], c["kc"].dtype
    live = (slots >= 0) & (slots < c["kc"].shape[0] * P)
    pg, row = slots[live] // P, slots[live] % P
    want, size = refs.rotate(k_in, c["pos"], c["freqs"], c["rot"], interleaved, mscale)
    for cch, w, sz, sc, old in ((c["kc"], want, size, c["ks"], before[0]),
                                (c["vc"], v_in.double(), torch.zeros_like(want), c["vs"], before[1])):
        w, sz = w[live] / sc, sz[live] / sc
        if cache == E4:
            w, sz = w.clamp(-448, 448), sz + w.abs() * refs.U32 / rel
        within(cch[pg, row], w, sz * rel, cache, what + " cache")
        now = raw(cch).clone()
        now[pg, row] = old[pg, row]
        assert torch.equal(now, old), what + ": other rows of the cache changed"
    return got


@pytest.mark.parametrize("T", [1, 2, 33, 700])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
def test_rope_types_and_lengths(cuda_device, T, interleaved, dtype, cache):
    rope_check(rope_case(cuda_device, T, 8, 2, 128, 128, dtype=dtype, cache=cache, seed=T), interleaved, what=f"T={T}")


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (64, 16), (64, 0), (80, 80), (80, 40), (96, 24), (256, 256), (512, 512),
                                   (6, 4), (7, 2), (33, 32), (130, 130), (100, 10), (1, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_head_sizes(cuda_device, D, rot, interleaved):
    for cache in (BF, E4):
        rope_check(rope_case(cuda_device, 9, 3, 1, D, rot, dtype=BF, cache=cache, seed=D + rot), interleaved, mscale=1.25,
                   what=f"D={D} rot={rot}")


def test_rope_far_positions(cuda_device):
    c = rope_case(cuda_device, 64, 4, 2, 64, 64, dtype=HF, seed=3, scaling="by_parts")
    c["pos"][:] = 2 ** 31 - 1 - torch.arange(64, device=cuda_device, dtype=torch.int32) * 7919
    c["pos"][:8] = torch.tensor([0, 1, 2, -1, -100000, -2 ** 31, 2 ** 30, 2 ** 20 + 1], dtype=torch.int32)
    # the reference's own angle (a 64-bit product, then a 64-bit cosine) is off
    # by 2^-53 * 2^31 radians, the kernel's by 2^-33 turns and by 2^31 * 2^-52
    # turns from its FP64 quotient: 2^-18 together
    q_in = c["q"].clone()
    got = moe.rope_append(c["q"], c["k"], c["v"], c["pos"], c["slots"], c["freqs"], c["kc"], c["vc"])
    want, size = refs.rotate(q_in, c["pos"], c["freqs"], 64, False, 1.0)
    within(got, want, size * (2.0 ** -18 + 2.0 ** -20), HF, "far")


def test_rope_layouts_padding_and_in_place(cuda_device):
    c = rope_case(cuda_device, 40, 4, 2, 64, 32, seed=4)
    c["kc"] = c["kc"].transpose(1, 2).contiguous().transpose(1, 2)     # heads before tokens
    c["vc"] = torch.cat((c["vc"], c["vc"]), -1)[..., 32:96]            # a slice of wider rows
    c["slots"][3] = -1
    c["slots"][7] = -12345
    rope_check(c, what="layouts")
    c = rope_case(cuda_device, 40, 4, 2, 64, 64, seed=5)
    before = c["q"].clone()
    got = rope_check(c, interleaved=True, q_out=c["q"], what="in place")
    assert got.data_ptr() == c["q"].data_ptr() and not torch.equal(got, before)
    c = rope_case(cuda_device, 5, 4, 2, 64, 64, seed=6)
    c["slots"][2] = c["kc"].shape[0] * c["kc"].shape[1]                # one past the cache
    c["slots"][4] = 2 ** 62
    rope_check(c, what="beyond")
    assert moe.device_error(cuda_device) & 0x8


def test_rope_unaligned_rows(cuda_device):
    c = rope_case(cuda_device, 11, 3, 1, 64, 64, seed=7)
    wide = torch.zeros(11, 5, 67, dtype=BF, device=cuda_device)
    wide[..., 1:65] = torch.cat((c["q"], c["k"], c["v"]), 1)
    c["q"], c["k"], c["v"] = wide[..., 1:65].split([3, 1, 1], 1)
    rope_check(c, what="unaligned")


def test_rope_e4m3_saturates_and_keeps_nan(cuda_device):
    c = rope_case(cuda_device, 2, 1, 1, 64, 64, cache=E4, seed=8)
    c["v"][0] = 1e4
    c["v"][1] = float("nan")
    c["vs"] = 0.5
    moe.rope_append(c["q"], c["k"], c["v"], c["pos"], c["slots"], c["freqs"], c["kc"], c["vc"], v_scale=0.5)
    rows = c["vc"].float().view(-1, 64)[c["slots"]]
    assert bool((rows[0] == 448).all()) and bool(torch.isnan(rows[1]).all())


# -------------------------------------------------------------------- norm ---

def norm_check(dev, T, d, dtype=BF, resid=None, post=None, pre="rms", gate="none", act="none", alpha=1.0, bias=False,
               seed=0, what="", std=1.0, cut=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    y = (rnd(T, d + cut) * std).to(dtype)[:, cut:]
    r = None if resid is None else (rnd(T, d + cut) * 3).to(resid)[:, cut:]
    gt = None if gate == "none" else rnd(*{"full": (T, d), "row": (T, 1), "column": (1, d), "one": (1, 1)}[gate]).to(dtype)

    def spec(kind):
        if kind is None:
            return None
        return moe.Norm((1 + 0.2 * rnd(d)).to(dtype) if kind != "bare" else None, rnd(d).to(dtype) if bias else None,
                        1e-5, "rms" if kind == "bare" else kind)

    sp, sq = spec(post), spec(pre)
    got = moe.norm_residual(y, r, post=sp, gate=gt, gate_act=act, alpha=alpha, pre=sq)
    torch.cuda.synchronize()
    (wr, er), (wx, ex) = refs.norm_residual(y, r, sp and tuple(sp), gt, act, alpha, sq and tuple(sq))
    if r is None:
        within(got, wx, ex, dtype, what + " x")
    else:
        within(got[0], wr, er, resid, what + " r")
        within(got[1], wx, ex, dtype, what + " x")


@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (2, 8), (5, 128), (1, 256), (7, 264), (2, 512), (3, 1000), (1, 1024), (4, 2048), (1, 2056),
                                 (3, 4096), (2, 7168), (1, 8200), (2, 16384), (1, 16392), (2, 20001), (1, 32768)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_sizes(cuda_device, T, d, kind):
    norm_check(cuda_device, T, d, BF, BF, pre=kind, seed=d, what=f"{T}x{d}")
    norm_check(cuda_device, T, d, HF, F32, post=kind, pre=kind, gate="full", act="sigmoid", alpha=-0.5, bias=True, seed=d,
               what=f"{T}x{d} full")


@pytest.mark.parametrize("d", [200, 201, 2048])
@pytest.mark.parametrize("gate", ["none", "full", "row", "column", "one"])
@pytest.mark.parametrize("act", ["none", "sigmoid"])
@pytest.mark.parametrize("resid", [None, BF, F32])
def test_norm_parts(cuda_device, d, gate, act, resid):
    for post in (None, "rms"):
        for pre in (None, "layer", "bare"):
            norm_check(cuda_device, 6, d, BF, resid, post, pre, gate, act, 0.25, bias=True, seed=d,
                       what=f"d={d} {gate} {act} {resid} {post} {pre}")


def test_norm_many_rows_and_slices(cuda_device):
    norm_check(cuda_device, 3001, 128, HF, HF, seed=1, what="rows")
    norm_check(cuda_device, 9, 256, BF, F32, post="rms", seed=2, cut=8, what="aligned slice")
    norm_check(cuda_device, 9, 256, BF, BF, post="rms", seed=3, cut=3, what="odd slice")


def test_norm_constant_and_zero_rows(cuda_device):
    y = torch.zeros(3, 512, dtype=BF, device=cuda_device)
    y[1] = 5.0
    for kind in ("rms", "layer"):
        x = moe.norm_residual(y, pre=moe.Norm(kind=kind))
        assert not bool(torch.isnan(x).any()) and int((x[0] != 0).sum()) == 0
        assert bool((x[1] == (1.0 if kind == "rms" else 0.0)).all())
    # a large mean over a small spread: centred squares, not moments
    y = (1000 + torch.arange(512, device=cuda_device) % 2 * 8).to(BF).repeat(2, 1)
    x = moe.norm_residual(y, pre=moe.Norm(kind="layer", eps=0.0))
    assert bool((x.abs() == 1.0).all())


def test_norm_in_place_and_graph(cuda_device):
    g = torch.Generator(device=cuda_device).manual_seed(5)
    y, r = (torch.randn(8, 2048, generator=g, device=cuda_device).to(BF) for _ in range(2))
    w = moe.Norm(torch.ones(2048, dtype=BF, device=cuda_device))
    wr, wx = moe.norm_residual(y, r, pre=w)
    r2, y2 = r.clone(), y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.norm_residual(y2, r2, pre=w, resid_out=r2, out=y2)
    r2.copy_(r), y2.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r2, wr) and torch.equal(y2, wx)


# ------------------------------------------------------------ 4-bit weights ---

def mv_check(dev, T, N, K, group, dtype=BF, zeros=True, seed=0, what="", pad=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(T, K + pad, generator=g, device=dev).to(dtype)[:, :K]
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    scales = (0.02 * torch.randn(N, K // group, generator=g, device=dev)).to(dtype)
    z = torch.randint(0, 16, (N, K // group), generator=g, device=dev, dtype=torch.uint8) if zeros else None
    guard = torch.full((T, N + 32), 7.0, dtype=dtype, device=dev)
    y = guard[:, 16:16 + N]
    moe.matvec4(x, moe.W4(codes, scales, z), y=y)
    torch.cuda.synchronize()
    want, bound = refs.matvec4(x, codes, scales, z, group)
    within(y, want, bound, dtype, what)
    assert bool((guard[:, :16] == 7).all()) and bool((guard[:, 16 + N:] == 7).all()), what + ": guard"


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 32, 33, 100, 256])
@pytest.mark.parametrize("dtype,group", [(BF, 32), (HF, 64), (BF, 128)])
def test_matvec_tokens(cuda_device, T, dtype, group):
    mv_check(cuda_device, T, 100, 384, group, dtype, seed=T, what=f"T={T}")


@pytest.mark.parametrize("N", [1, 15, 16, 17, 33, 1000, 9729, 9745])
@pytest.mark.parametrize("group", [32, 128])
def test_matvec_rows(cuda_device, N, group):
    for T in (1, 12):
        mv_check(cuda_device, T, N, 256, group, BF, seed=N, what=f"N={N}")


@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (96, 32), (64, 64), (128, 128), (1184, 32), (2048, 64), (2176, 64),
                                     (4224, 128), (20000, 32), (16384, 128)])
@pytest.mark.parametrize("zeros", [False, True])
def test_matvec_depths(cuda_device, K, group, zeros):
    mv_check(cuda_device, 1, 70, K, group, HF, zeros, seed=K, what=f"K={K}")
    mv_check(cuda_device, 5, 10000, K if K < 5000 else 512, group if K < 5000 else 32, BF, zeros, seed=K, what=f"K={K} wide")


def test_matvec_every_code_and_zero(cuda_device):
    """One-hot rows of x read back each weight: exact in FP16 (scale 1)."""
    K = 64
    codes = torch.arange(256, dtype=torch.uint8, device=cuda_device)[:, None].expand(256, K // 2).contiguous()
    z = (torch.arange(256, device=cuda_device) % 16).to(torch.uint8)[:, None].expand(256, 2).contiguous()
    scales = torch.ones(256, 2, dtype=HF, device=cuda_device)
    y = moe.matvec4(torch.eye(K, dtype=HF, device=cuda_device), moe.W4(codes, scales, z))
    c = torch.stack((codes & 15, codes >> 4), -1).view(256, K).float()
    assert torch.equal(y.T.float(), c - z.float()[:, :1])


def test_matvec_strided_x_and_graph(cuda_device):
    mv_check(cuda_device, 6, 50, 256, 64, seed=1, pad=24, what="strided")
    x = torch.randn(1, 512, device=cuda_device).to(BF)
    w = moe.W4(torch.randint(0, 256, (64, 256), device=cuda_device, dtype=torch.uint8),
               torch.rand(64, 4, device=cuda_device).to(BF))
    want = moe.matvec4(x, w)
    y = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.matvec4(x, w, y=y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and math.isfinite(float(y.float().sum()))


@pytest.mark.parametrize("dtype,T", [(BF, 1), (BF, 3), (BF, 8), (HF, 1), (HF, 2), (HF, 4)])
def test_matvec_few_rows_single_weights(cuda_device, dtype, T):
    """One element of x per row, all its significant bits set: each output is one weight times it, rounded once."""
    K, N = 96, 256
    codes = torch.arange(256, dtype=torch.uint8, device=cuda_device)[:, None].expand(256, K // 2).contiguous()
    z = (torch.arange(256, device=cuda_device) % 16).to(torch.uint8)[:, None].expand(256, 3).contiguous()
    scales = torch.ones(256, 3, dtype=dtype, device=cuda_device)
    full = 2 - torch.finfo(dtype).eps     # every bit of the significand
    for k in (0, 1, 31, 32, 77, 95):
        x = torch.zeros(T, K, dtype=dtype, device=cuda_device)
        for t in range(T):
            x[t, (k + 5 * t) % K] = full * 2.0 ** (3 * t - 9) * (-1) ** t
        y = moe.matvec4(x, moe.W4(codes, scales, z))
        for t in range(T):
            kk = (k + 5 * t) % K
            w = (codes[:, 0] >> (4 * (kk % 2)) & 15).double() - z[:, 0].double()
            assert torch.equal(y[t], (w * x[t, kk].double()).to(dtype)), (k, t)
    assert int((moe.matvec4(torch.zeros(T, K, dtype=dtype, device=cuda_device), moe.W4(codes, scales, z)) != 0).sum()) == 0


@pytest.mark.parametrize("dtype", [BF, HF])
def test_matvec_few_rows_of_wide_range(cuda_device, dtype):
    """Elements over 24 binades in one row, and rows of very different size.  An element's parts are exact down to
    2^-13 of its row's largest and within 2^-22 of the largest below: that much, times the weights, beside FP32."""
    g = torch.Generator(device=cuda_device).manual_seed(3)
    N, K, group = 130, 1024, 64
    for rows in ((1.0,), (1.0, 2.0 ** -8), (2.0 ** 6, 2.0 ** -2, 1.0, 2.0 ** -6)):
        x = torch.randn(len(rows), K, generator=g, device=cuda_device) * torch.tensor(rows, device=cuda_device)[:, None]
        x = (x * 2.0 ** -torch.randint(0, 25, x.shape, generator=g, device=cuda_device).float()).to(dtype)
        codes = torch.randint(0, 256, (N, K // 2), generator=g, device=cuda_device, dtype=torch.uint8)
        scales = torch.rand(N, K // group, generator=g, device=cuda_device).to(dtype)
        y = moe.matvec4(x, moe.W4(codes, scales))
        want, bound = refs.matvec4(x, codes, scales, None, group)
        weights = 15 * scales.double().repeat_interleave(group, 1).sum(1)
        within(y, want, bound + 2.0 ** -22 * x.double().abs().amax(1, keepdim=True) * weights, dtype, "wide range")


@pytest.mark.parametrize("K,group", [(32, 32), (96, 32), (128, 64), (128, 128), (1184, 32), (2176, 64), (4224, 128), (20000, 32)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_matvec_one_row_many_weights(cuda_device, K, group, dtype):
    mv_check(cuda_device, 1, 9729, K, group, dtype, K % 64 == 0, seed=K, what=f"K={K}")


@pytest.mark.parametrize("dtype", [BF, HF])
def test_matvec_one_row_single_weights_and_wide_range(cuda_device, dtype):
    """As the tests of few rows, with the weight rows for which a single row of x is split into 8-bit parts."""
    K, N = 96, 9984
    codes = torch.arange(N, device=cuda_device).to(torch.uint8)[:, None].expand(N, K // 2).contiguous()
    z = (torch.arange(N, device=cuda_device) % 16).to(torch.uint8)[:, None].expand(N, 3).contiguous()
    scales = torch.ones(N, 3, dtype=dtype, device=cuda_device)
    full = 2 - torch.finfo(dtype).eps
    for k, size in ((0, 1.0), (31, 2.0 ** -9), (32, -2.0 ** 12), (95, 3 * 2.0 ** -14)):
        x = torch.zeros(1, K, dtype=dtype, device=cuda_device)
        x[0, k] = full * size if size != 3 * 2.0 ** -14 else size
        w = (codes[:, 0] >> (4 * (k % 2)) & 15).double() - z[:, 0].double()
        y = moe.matvec4(x, moe.W4(codes, scales, z))
        assert torch.equal(y[0], (w * x[0, k].double()).to(dtype)), k
    assert int((moe.matvec4(torch.zeros(1, K, dtype=dtype, device=cuda_device), moe.W4(codes, scales, z)) != 0).sum()) == 0
    g = torch.Generator(device=cuda_device).manual_seed(4)
    K, group = 1024, 64
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=cuda_device, dtype=torch.uint8)
    scales = torch.rand(N, K // group, generator=g, device=cuda_device).to(dtype)
    weights = 15 * scales.double().repeat_interleave(group, 1).sum(1)
    for top in (1.0, 2.0 ** 10, 2.0 ** -4):
        x = torch.randn(1, K, generator=g, device=cuda_device)
        x = (x * top * 2.0 ** -torch.randint(0, 25, x.shape, generator=g, device=cuda_device).float()).to(dtype)
        want, bound = refs.matvec4(x, codes, scales, None, group)
        bound = bound + 2.0 ** -22 * x.double().abs().max() * weights
        y = moe.matvec4(x, moe.W4(codes, scales))
        # (FP16 at the largest size passes the type's range in places: infinite there)
        most = torch.finfo(dtype).max
        inside, beyond = want.abs() + bound < most, want.abs() - bound > most * (1 + refs.half_step(dtype))
        within(y[inside], want[inside], bound[inside], dtype, "wide")
        assert torch.equal(y[beyond].double(), want[beyond].sign() * math.inf)


@pytest.mark.parametrize("T,d", [(1, 9), (2, 1), (9, 15), (17, 85), (8, 255), (1300, 257), (5, 505), (1300, 511), (3, 1017), (4, 2041), (3, 4095),
                                 (2, 8183), (3, 8185), (2, 16375), (2, 16377), (11, 340)])
@pytest.mark.parametrize("gate", ["none", "full", "column", "row"])
def test_norm_rows_between_vectors(cuda_device, T, d, gate):
    for resid in (BF, F32):
        norm_check(cuda_device, T, d, BF, resid, "layer", "rms", gate, "sigmoid", 0.5, bias=True, seed=d, what=f"{T}x{d} {gate}")
    # nothing beyond the arrays' ends is written
    y = torch.randn(T * d + 64, device=cuda_device).to(HF)
    buf = [torch.full((T * d + 64,), 7.0, dtype=HF, device=cuda_device) for _ in range(2)]
    inner = [b[32:32 + T * d].view(T, d) for b in buf]
    moe.norm_residual(y[:T * d].view(T, d), y[:T * d].view(T, d), pre=moe.Norm(), resid_out=inner[0], out=inner[1])
    for b in buf:
        assert bool((b[:32] == 7).all()) and bool((b[32 + T * d:] == 7).all())
    # in place, a row's end next to another row's beginning
    r = y[:T * d].view(T, d).clone()
    want, x = moe.norm_residual(y[:T * d].view(T, d), r, pre=moe.Norm())
    moe.norm_residual(y[:T * d].view(T, d), r, pre=moe.Norm(), resid_out=r)
    assert torch.equal(r, want)


@pytest.mark.parametrize("N,K,group", [(77900, 256, 128), (77825, 32, 32), (38950, 512, 64), (38920, 416, 32), (19470, 1024, 128),
                                       (19457, 800, 32), (19500, 2304, 64), (9730, 2048, 32), (9731, 6016, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_matvec_one_row_short_and_uneven_depths(cuda_device, N, K, group, dtype):
    """Block tiles of several warps' rows (fewer than eight steps of K, or steps that do not divide by eight)."""
    mv_check(cuda_device, 1, N, K, group, dtype, True, seed=K, what=f"{N}x{K}")
    mv_check(cuda_device, 3, N // 4 + 1, K, group, dtype, False, seed=K, what=f"3 rows, {N // 4 + 1}x{K}")
