"""GPU parity of moe_paged_attention against a plain implementation in 64 bits, with bounds derived in _block_refs."""
import math

import pytest
import torch

import mixture_experts_decode_gb300 as moe
import _block_refs as refs

pytestmark = pytest.mark.gpu
BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def make(dev, lens, Hq, Hkv, D, page, dtype=BF, cache=None, seed=0, order="nhd", spare=2, q_std=1.5):
    g = torch.Generator(device=dev).manual_seed(seed)
    cache = cache or dtype
    used = [-(-max(n, 0) // page) for n in lens]
    most, pages = max(used + [1]), sum(used) + spare
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), most), -7, dtype=torch.int32)
    for b, u in enumerate(used):
        for i in range(u):
            table[b, i] = perm.pop()
    shape = (pages, page, Hkv, D) if order == "nhd" else (pages, Hkv, page, D)
    ks, vs = (0.03, 0.02) if cache == E4 else (1.0, 1.0)
    rnd = lambda sc: (torch.randn(shape, generator=g, device=dev) / sc).to(cache)  # noqa: E731
    k, v = rnd(ks), rnd(vs)
    if order == "hnd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    q = (torch.randn(len(lens), Hq, D, generator=g, device=dev) * q_std).to(dtype)
    return dict(q=q, k=k, v=v, table=table.to(dev), lens=torch.tensor(lens, dtype=torch.int32, device=dev), ks=ks, vs=vs)


def check(c, window=0, sinks=0, scale=None, ws=None, what=""):
    q = c["q"]
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out, lse = moe.paged_attention(q, c["k"], c["v"], c["table"], c["lens"], scale=scale, window=window, sinks=sinks,
                                   k_scale=c["ks"], v_scale=c["vs"], workspace=ws, return_lse=True)
    torch.cuda.synchronize()
    ro, rl, ob, lb = refs.attention(q, c["k"], c["v"], c["table"], c["lens"], scale, window, sinks, c["ks"], c["vs"])
    assert out.dtype == q.dtype and not torch.isnan(out).any(), what
    err = (out.double() - ro).abs() - ob
    assert err.max() <= 0, f"{what}: out beyond its bound by {err.max().item():.3g}"
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty), what
    e = ((lse.double() - rl).abs() - lb)[~empty]
    assert e.numel() == 0 or e.max() <= 0, f"{what}: lse beyond its bound by {e.max().item():.3g}"
    return out, lse


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 200])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
def test_short_lengths(cuda_device, n, dtype, cache):
    check(make(cuda_device, [n], 8, 2, 64, 16, dtype, cache, seed=n), what=f"n={n}")


@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 144, 192, 256])
@pytest.mark.parametrize("cache", [BF, E4])
def test_head_sizes(cuda_device, D, cache):
    check(make(cuda_device, [70, 0, 333], 6, 3, D, 24, BF, cache, seed=D), what=f"D={D}")


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 1), (9, 1), (16, 1), (17, 1), (20, 1), (40, 8), (64, 4), (128, 1)])
@pytest.mark.parametrize("cache", [HF, E4])
def test_head_groups(cuda_device, Hq, Hkv, cache):
    check(make(cuda_device, [100, 37], Hq, Hkv, 64, 16, HF, cache, seed=Hq), what=f"{Hq}/{Hkv}")


@pytest.mark.parametrize("D,cache", [(128, E4), (256, BF), (256, E4), (128, BF)])
def test_wide_groups_of_wide_heads(cuda_device, D, cache):
    check(make(cuda_device, [517, 64], 16, 1, D, 32, BF, cache, seed=D), what=f"D={D}")


@pytest.mark.parametrize("page", [1, 3, 8, 13, 16, 100, 256])
def test_page_sizes(cuda_device, page):
    check(make(cuda_device, [1, 99, 100, 101, 257], 4, 2, 128, page, BF, seed=page), what=f"page={page}")


@pytest.mark.parametrize("cache", [BF, E4])
def test_ragged_batch_cut_over_blocks(cuda_device, cache):
    lens = [3000, 1, 0, 17, 900, 64, 128, 5000, 0, 33]
    check(make(cuda_device, lens, 16, 4, 128, 64, BF, cache, seed=5), what="ragged")


def test_more_sequences_than_blocks(cuda_device):
    lens = [(i * 37) % 90 for i in range(700)]
    check(make(cuda_device, lens, 2, 1, 64, 16, HF, seed=6), what="700 sequences")


def test_one_long_sequence(cuda_device):
    check(make(cuda_device, [40000], 8, 1, 128, 128, BF, seed=7, q_std=3.0), what="long")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (63, 5), (64, 64), (100, 3), (1000, 4), (10, 1000)])
@pytest.mark.parametrize("cache", [BF, E4])
def test_window_and_sinks(cuda_device, window, sinks, cache):
    c = make(cuda_device, [1, 5, 64, 101, 350, 1200], 8, 2, 64, 24, BF, cache, seed=window)
    check(c, window, sinks, what=f"window={window} sinks={sinks}")


def test_unseen_tokens_are_not_read(cuda_device):
    c = make(cuda_device, [300], 8, 2, 64, 16, BF, seed=8)
    want, _ = check(c, window=50, sinks=3)
    seen = set(refs.visible(300, 50, 3))
    tab = c["table"].cpu()
    kept = {(int(tab[0, j // 16]), j % 16) for j in seen}
    for pg in range(c["k"].shape[0]):
        for row in range(16):
            if (pg, row) not in kept:
                c["k"][pg, row] = float("nan")
                c["v"][pg, row] = float("inf")
    for i in range(tab.shape[1]):
        if not any(j // 16 == i for j in seen):
            c["table"][0, i] = 1 << 30      # never looked up either
    got = moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], window=50, sinks=3)
    assert torch.equal(got, want)


@pytest.mark.parametrize("cache", [BF, E4])
def test_strides_and_layouts(cuda_device, cache):
    lens = [90, 41]
    c = make(cuda_device, lens, 8, 4, 64, 16, BF, cache, seed=9, order="hnd")
    assert not c["k"].is_contiguous()
    check(c, what="heads before tokens")
    # keys and values side by side in one buffer, q and the table as slices of wider ones
    kv = torch.stack((c["k"], c["v"]), 3).contiguous()
    wide_q = torch.zeros(2, 8, 160, dtype=BF, device=cuda_device)
    wide_q[..., 16:80] = c["q"]
    wide_t = torch.full((2, 40), -1, dtype=torch.int32, device=cuda_device)
    wide_t[:, 3:3 + c["table"].shape[1]] = c["table"]
    d = dict(c, k=kv[:, :, :, 0], v=kv[:, :, :, 1], q=wide_q[..., 16:80], table=wide_t[:, 3:3 + c["table"].shape[1]])
    check(d, what="strided")


def test_scales_and_extremes(cuda_device):
    c = make(cuda_device, [200], 8, 2, 128, 16, BF, E4, seed=10)
    check(c, scale=-0.2, what="negative scale")
    check(c, scale=0.0, what="scale 0 (a plain mean)")
    c["q"] = c["q"] * 1e-6
    check(c, what="tiny q")
    c["q"] = (c["q"].double() * 1e6 * 1e4).to(BF)   # scores of tens of thousands: one key takes all
    out, _ = moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], k_scale=c["ks"], v_scale=c["vs"],
                                 return_lse=True)
    assert torch.isfinite(out).all()


def test_long_tail_below_the_maximum(cuda_device):
    """One key far above 30000 others that hold a share of the weight together."""
    n, D = 30000, 64
    c = make(cuda_device, [n], 1, 1, D, 64, HF, E4, seed=11)
    c["q"].zero_()
    c["q"][0, 0, 0] = 1.0
    k, v = c["k"].view(torch.uint8), c["v"].view(torch.uint8)
    k.zero_()
    v.zero_()
    v.copy_(torch.full_like(c["v"], 0, dtype=torch.float16).add_(1.0).to(E4).view(torch.uint8))
    first = int(c["table"][0, 0])
    c["k"].view(torch.uint8)[first, 0, 0, 0] = torch.tensor(352.0).to(E4).view(torch.uint8).item()
    c["v"].view(torch.uint8)[first, 0] = 0
    c["ks"], c["vs"] = 1.0, 1.0
    # e^12 = 162754 against 29999 keys of weight 1: 0.1556 of the mass
    out, _ = check(c, scale=12.0 / 352.0, what="tail")
    assert abs(out[0, 0, 5].item() - 29999 / (29999 + math.exp(12))) < 1e-3
    # e^18: each of the others weighs 2^-26 of the largest
    out, _ = check(c, scale=18.0 / 352.0, what="far tail")
    want = 29999 / (29999 + math.exp(18))
    assert abs(out[0, 0, 5].item() - want) < 2e-3 * want


def test_inf_and_nan_keys_stay_in_their_rows(cuda_device):
    c = make(cuda_device, [50, 50], 4, 2, 64, 16, BF, seed=12)
    want = moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"])
    c["v"][int(c["table"][1, 0]), 3] = float("nan")
    got = moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"])
    assert torch.equal(got[0], want[0]) and torch.isnan(got[1]).all()


def test_workspace_is_left_clean_and_reused(cuda_device):
    ws = moe.attention_workspace(64, 1, 256, cuda_device)
    for Hq, Hkv, D, lens in ((8, 2, 64, [5000, 70]), (16, 1, 256, [9000]), (64, 4, 128, [33] * 40), (8, 2, 64, [12000])):
        c = make(cuda_device, lens, Hq, Hkv, D, 64, BF, seed=D)
        a, _ = check(c, ws=ws, what="kept workspace")
        assert int(ws[:2048].max()) == 0
        b, _ = check(c, ws=ws, what="again")
        assert torch.equal(a, b)     # the join's order is fixed


def test_streams_and_graphs(cuda_device):
    c = make(cuda_device, [2000, 300], 8, 2, 128, 64, BF, seed=13)
    ws = moe.attention_workspace(8, 2, 128, cuda_device)
    out = torch.empty_like(c["q"])
    want, _ = check(c, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], workspace=ws, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], workspace=ws, out=out)
    for lens in ([2000, 300], [17, 0], [1999, 1]):
        c["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"])), lens


def test_bad_pages_and_lengths_are_left_out(cuda_device):
    c = make(cuda_device, [100, 60], 8, 2, 64, 16, BF, seed=14)
    c["table"][0, 2] = c["k"].shape[0]          # one past the cache
    c["table"][0, 4] = -1
    check(c, what="bad pages")
    assert moe.device_error(cuda_device) & 0x8
    c["table"][:] = -1
    out, lse = moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], return_lse=True)
    assert int((out != 0).sum()) == 0 and bool((lse == -math.inf).all())
    assert moe.device_error(cuda_device) & 0x8
    c = make(cuda_device, [100, 60], 8, 2, 64, 16, BF, seed=14)
    cap = c["table"].shape[1] * 16
    c["lens"].copy_(torch.tensor([cap + 1000, -5], dtype=torch.int32))
    check(c, what="bad lengths")
    assert moe.device_error(cuda_device) & 0x8


def test_dirty_counters_are_reported(cuda_device):
    c = make(cuda_device, [5000], 8, 1, 64, 64, BF, seed=15)
    ws = moe.attention_workspace(8, 1, 64, cuda_device)
    ws[:2048] = 77
    moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], workspace=ws)
    assert moe.device_error(cuda_device) & 0x10


def test_outputs_stay_in_bounds(cuda_device):
    c = make(cuda_device, [70, 0, 300], 5, 1, 80, 16, BF, seed=16)
    buf = torch.full((3 * 5 * 80 + 256,), 7.0, dtype=BF, device=cuda_device)
    lbuf = torch.full((15 + 64,), 7.0, device=cuda_device)
    need = moe.attention_workspace_bytes(5, 1, 80)
    ws = torch.zeros(need + 512, dtype=torch.uint8, device=cuda_device)
    ws[need:] = 99
    moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], workspace=ws[:need],
                        out=buf[128:-128].view(3, 5, 80), lse=lbuf[32:-32].view(3, 5))
    torch.cuda.synchronize()
    assert bool((buf[:128] == 7).all()) and bool((buf[-128:] == 7).all()) and not bool((buf[128:-128] == 7).all())
    assert bool((lbuf[:32] == 7).all()) and bool((lbuf[-32:] == 7).all())
    assert bool((ws[need:] == 99).all())


def test_cache_beyond_32_bit_offsets(cuda_device):
    """Page offsets past 2^31 elements (a page stride of 2^21 elements, 1200 pages, views of one buffer)."""
    P, Hkv, D, stride = 16, 2, 64, 1 << 21
    pages = 1200
    raw = torch.zeros(pages * stride, dtype=torch.uint8, device=cuda_device).view(E4)
    k = raw.as_strided((pages, P, Hkv, D), (stride, Hkv * D, D, 1))
    v = raw.as_strided((pages, P, Hkv, D), (stride, Hkv * D, D, 1), P * Hkv * D)
    g = torch.Generator(device=cuda_device).manual_seed(17)
    chosen = [1199, 1100, 3, 1024, 1025]
    for pg in chosen:
        k[pg].view(torch.uint8).copy_((torch.randn(P, Hkv, D, generator=g, device=cuda_device) * 20).to(E4).view(torch.uint8))
        v[pg].view(torch.uint8).copy_((torch.randn(P, Hkv, D, generator=g, device=cuda_device) * 20).to(E4).view(torch.uint8))
    q = torch.randn(1, 4, D, generator=g, device=cuda_device).to(BF)
    c = dict(q=q, k=k, v=v, table=torch.tensor([chosen], dtype=torch.int32, device=cuda_device),
             lens=torch.tensor([75], dtype=torch.int32, device=cuda_device), ks=0.05, vs=0.05)
    check(c, what="far pages")


def test_empty_batch(cuda_device):
    c = make(cuda_device, [5], 4, 2, 64, 16, BF, seed=18)
    out = moe.paged_attention(c["q"][:0], c["k"], c["v"], c["table"][:0], c["lens"][:0])
    assert out.shape == (0, 4, 64)


def test_cache_without_pages(cuda_device):
    q = torch.randn(2, 4, 64, device=cuda_device).to(BF)
    empty = torch.zeros(0, 16, 2, 64, dtype=BF, device=cuda_device)
    table = torch.zeros(2, 3, dtype=torch.int32, device=cuda_device)
    lens = torch.tensor([5, 0], dtype=torch.int32, device=cuda_device)
    out, lse = moe.paged_attention(q, empty, empty, table, lens, return_lse=True)
    assert int((out != 0).sum()) == 0 and bool((lse == -math.inf).all())
    assert moe.device_error(cuda_device) & 0x8


def test_output_over_the_query(cuda_device):
    c = make(cuda_device, [3000, 40, 0, 700], 20, 1, 128, 64, BF, seed=19)
    want, _ = check(c)
    moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], out=c["q"])
    assert torch.equal(c["q"], want)
