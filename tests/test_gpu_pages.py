"""moe_plan_pages and moe_release_pages against the same bookkeeping request by request on the host (all exact)."""
import pytest
import torch

import mixture_experts_decode_gb300 as moe
import _serving_refs as refs

pytestmark = pytest.mark.gpu
POOL = 0x20


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0


def i32(dev, v):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def check_plan(dev, past, new, table, free, n_free, page, T, shared=(), shares=None, in_place=False, stride=0, offset=0):
    B, most = len(past), len(table[0]) if table else 0
    wide = torch.full((B, most + stride), -99, dtype=torch.int32, device=dev)
    tab = wide[:, :most]
    if B:
        tab.copy_(i32(dev, table).view(B, most))
    lens, height = i32(dev, past), i32(dev, [n_free])
    kw = dict(seq_lens=lens, n_free_out=height) if in_place else {}
    bufs = [torch.full((T + 8,), -77, dtype=t, device=dev) for t in (torch.int32, torch.int64, torch.int32)]
    outs = [b[offset:offset + T] for b in bufs]
    stack = i32(dev, free)
    got = moe.plan_pages(lens, i32(dev, new), tab, stack, height, page, T,
                         shared_pages=i32(dev, list(shared)) if shared else None,
                         shares=None if shares is None else torch.tensor(shares, dtype=torch.bool, device=dev),
                         positions=outs[0], slots=outs[1], seq_ids=outs[2], **kw)
    torch.cuda.synchronize()
    pos, slots, seqs, starts, rlens, left, rtab, refused = refs.plan(past, new, table, free, n_free, page, T, list(shared),
                                                                     shares)
    assert got.starts.tolist() == starts
    assert got.positions.tolist() == pos and got.slots.tolist() == slots and got.seq_ids.tolist() == seqs
    assert got.seq_lens.tolist() == rlens and got.n_free.tolist() == [left]
    assert tab.tolist() == rtab and stack.tolist() == list(free)
    assert bool((wide[:, most:] == -99).all())
    for b in bufs:
        assert bool((b[:offset] == -77).all()) and bool((b[offset + T:] == -77).all())
    if not in_place:
        assert lens.tolist() == past and height.tolist() == [n_free]
    assert (moe.device_error(dev) == POOL) == refused
    return got, tab


@pytest.mark.parametrize("B", [0, 1, 2, 31, 64, 513, 1000, 4096])
@pytest.mark.parametrize("page", [1, 7, 16])
def test_random_states(cuda_device, B, page):
    g = torch.Generator().manual_seed(B * 100 + page)
    most = 40
    for new_max, in_place, ns in ((1, True, 0), (20, False, 3), (60, True, 2)):
        if B * new_max * (1 if page > 1 else 2) > 150000:
            new_max = 30
        past, new, table, free, n_free, shared, shares = refs.random_plan(g, B, page, most, 20, new_max, 1.0, ns)
        check_plan(cuda_device, past, new, table, free, n_free, page, sum(new) + 13, shared, shares, in_place, stride=3)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("room,cut", [(0.6, 0), (1.0, 50), (0.0, 0), (1.0, 100000)])
def test_refusals_of_pages_tokens_and_rows(cuda_device, room, cut, in_place):
    g = torch.Generator().manual_seed(3)
    past, new, table, free, n_free, shared, shares = refs.random_plan(g, 200, 8, 12, 90, 40, room, 0)
    past[17], new[40] = -1, -5
    check_plan(cuda_device, past, new, table, free, n_free, 8, max(0, sum(new) - cut), in_place=in_place)


def test_no_tokens_no_requests_no_pages(cuda_device):
    check_plan(cuda_device, [], [], [], [1, 2], 2, 4, 0)
    check_plan(cuda_device, [], [], [], [1, 2], 2, 4, 5)
    check_plan(cuda_device, [3, 0], [0, 0], [[0], [1]], [], 0, 4, 0)
    check_plan(cuda_device, [3, 0], [1, 0], [[0], [1]], [], 0, 4, 3)
    check_plan(cuda_device, [3, 0], [1, 1], [[0], [-1]], [], 0, 4, 3)     # refused: no page left


def test_unaligned_outputs(cuda_device):
    g = torch.Generator().manual_seed(4)
    past, new, table, free, n_free, shared, shares = refs.random_plan(g, 30, 16, 20, 100, 200, 1.0, 4)
    for offset in (1, 2, 3):
        check_plan(cuda_device, past, new, table, free, n_free, 16, sum(new), shared, shares, offset=offset)


def test_many_tokens_at_once(cuda_device):
    """Prompts of some hundred thousand tokens, over several blocks, in place and not."""
    g = torch.Generator().manual_seed(5)
    past, new, table, free, n_free, shared, shares = refs.random_plan(g, 60, 16, 700, 200, 10000, 1.0, 10)
    for in_place in (False, True):
        check_plan(cuda_device, past, new, table, free, n_free, 16, sum(new) + 5, shared, shares, in_place)


def test_lengths_near_the_largest(cuda_device):
    top = 2 ** 31 - 1
    check_plan(cuda_device, [top - 3, top - 1, top], [2, 3, 0], [[5, 6]] * 3, [9, 8], 2, 2 ** 30, 9)


def test_lengths_whose_sum_passes_32_bits(cuda_device):
    top = 2 ** 31 - 1
    for page in (1, 2, 7):
        check_plan(cuda_device, [0, top, 0, top - 1], [2, top, 2, top], [[5, 6]] * 4, [9, 8, 3], 3, page, 9)


def test_slots_past_32_bits(cuda_device):
    top = 2 ** 31 - 1
    check_plan(cuda_device, [0, 70, 64], [100, 3, 1], [[-1, -1], [top - 7, top - 8], [5, -1]], [9, 8, top - 3, top, top - 1], 5, 64, 110)


def test_a_stack_height_out_of_range_is_cut(cuda_device):
    for n, ok in ((-3, 0), (5, 2)):
        got = moe.plan_pages(i32(cuda_device, [0, 0]), i32(cuda_device, [1, 1]), i32(cuda_device, [[-1], [-1]]),
                             i32(cuda_device, [7, 4]), i32(cuda_device, [n]), 4, 2)
        assert moe.device_error(cuda_device) == POOL
        assert got.slots.tolist() == ([16, 28] if ok else [-1, -1]) and got.n_free.tolist() == [0]


def test_an_entry_below_zero_gives_no_slot(cuda_device):
    got = moe.plan_pages(i32(cuda_device, [3, 5]), i32(cuda_device, [1, 1]), i32(cuda_device, [[-1, -1], [2, 3]]),
                         i32(cuda_device, [7]), i32(cuda_device, [1]), 4, 2)
    assert got.slots.tolist() == [-1, 13]
    assert moe.device_error(cuda_device) == 0x8


@pytest.mark.parametrize("B", [0, 1, 33, 700, 4096])
@pytest.mark.parametrize("in_place", [False, True])
def test_release(cuda_device, B, in_place):
    dev = cuda_device
    g = torch.Generator().manual_seed(B)
    for page, ns in ((1, 0), (16, 3), (24, 50)):
        past, _, table, free, _, _, shares = refs.random_plan(g, B, page, 41, 40 * page, 0, 1.0, 0)
        ended = (torch.rand(B, generator=g) < 0.6).tolist()
        stack = free + [-55] * (41 * B + 4)
        d_stack, lens, height = i32(dev, stack), i32(dev, past), i32(dev, [len(free)])
        tab = i32(dev, table).view(B, 41)
        kw = dict(seq_lens_out=lens, n_free_out=height) if in_place else {}
        rl, rn = moe.release_pages(tab, lens, torch.tensor(ended, dtype=torch.bool, device=dev), d_stack, height, page, ns,
                                   torch.tensor(shares, dtype=torch.bool, device=dev), **kw)
        wf, wn, wl = refs.release(table, past, ended, stack, len(free), page, ns, shares)
        assert rl.tolist() == wl and rn.tolist() == [wn] and d_stack.tolist() == wf
        if not in_place:
            assert lens.tolist() == past and height.tolist() == [len(free)]


def test_release_beyond_the_stack_and_the_row(cuda_device):
    dev = cuda_device
    stack = i32(dev, [1, 2, -55, -55, -55])
    rl, rn = moe.release_pages(i32(dev, [[3, 4], [5, 6], [7, 8]]), i32(dev, [8, 4, 8]), torch.ones(3, dtype=torch.uint8, device=dev),
                               stack, i32(dev, [2]), 4)
    assert stack.tolist() == [1, 2, 3, 4, 5] and rn.tolist() == [5] and rl.tolist() == [0, 0, 0]
    assert moe.device_error(dev) == POOL
    stack = i32(dev, [-55] * 6)
    rl, rn = moe.release_pages(i32(dev, [[3, 4], [5, 6]]), i32(dev, [99, -2]), torch.ones(2, dtype=torch.uint8, device=dev),
                               stack, i32(dev, [0]), 4)
    assert stack.tolist() == [3, 4, -55, -55, -55, -55] and rn.tolist() == [2] and rl.tolist() == [0, 0]
    assert moe.device_error(dev) == POOL


def test_a_captured_step_runs_on(cuda_device):
    """Requests grow a token a step by replays of one graph, end, give their pages back and begin again."""
    dev, page, most, B = cuda_device, 4, 12, 6
    pool = B * most
    free = torch.randperm(pool, generator=torch.Generator().manual_seed(1)).tolist()
    lens, height, stack = i32(dev, [0] * B), i32(dev, [pool]), i32(dev, free)
    tab = torch.full((B, most), -1, dtype=torch.int32, device=dev)
    ones, ended = i32(dev, [1] * B), torch.zeros(B, dtype=torch.bool, device=dev)

    def step():
        moe.release_pages(tab, lens, ended, stack, height, page, seq_lens_out=lens, n_free_out=height)
        return moe.plan_pages(lens, ones, tab, stack, height, page, B + 2, seq_lens=lens, n_free_out=height)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = step()
    h_lens, h_tab, h_stack, h_free = [0] * B, tab.tolist(), list(free), pool
    g = torch.Generator().manual_seed(2)
    for i in range(60):
        e = (torch.rand(B, generator=g) < 0.1).tolist()
        ended.copy_(torch.tensor(e))
        h_stack, h_free, h_lens = refs.release(h_tab, h_lens, e, h_stack, h_free, page)
        pos, slots, seqs, starts, h_lens, h_free, h_tab, refused = refs.plan(h_lens, [1] * B, h_tab, h_stack, h_free, page, B + 2)
        graph.replay()
        torch.cuda.synchronize()
        assert (p.positions.tolist(), p.slots.tolist(), p.seq_ids.tolist(), p.starts.tolist()) == (pos, slots, seqs, starts), i
        assert lens.tolist() == h_lens and height.tolist() == [h_free] and tab.tolist() == h_tab, i
        assert stack.tolist() == h_stack, i
        used = [pg for b in range(B) for pg in h_tab[b][:-(-h_lens[b] // page)]]
        assert sorted(used + h_stack[:h_free]) == list(range(pool))      # no page lost or held twice
        assert (moe.device_error(dev) == POOL) == refused
