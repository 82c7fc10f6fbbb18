"""Infinities and NaN among the visible keys and values of moe_paged_attention."""
import math

import pytest
import torch

import mixture_experts_decode_gb300 as moe
from test_gpu_attention import BF, E4, HF, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0


def run(c):
    return moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], k_scale=c["ks"], v_scale=c["vs"], return_lse=True)


def at(c, b, tok):
    page = c["k"].shape[1]
    return int(c["table"][b, tok // page]), tok % page


@pytest.mark.parametrize("cache,bad", [(BF, math.inf), (BF, math.nan), (HF, -math.inf), (HF, math.nan), (E4, math.nan)])
@pytest.mark.parametrize("n,tok", [(50, 3), (3000, 2999), (3000, 0)])
def test_values_show_in_their_own_dim(cuda_device, cache, bad, n, tok):
    """No output of that key-value head's dim is finite; the other dims, heads and sequences are as they were."""
    c = make(cuda_device, [n, 77], 8, 2, 64, 16, cache if cache != E4 else BF, cache, seed=n)
    want, lse = run(c)
    pg, row = at(c, 0, tok)
    c["v"][pg, row, 1, 9] = bad
    got, lse2 = run(c)
    assert not bool(torch.isfinite(got[0, 4:, 9]).any())
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[0, 4:, 9] = False
    assert torch.equal(got[keep], want[keep]) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n", [50, 3000])
def test_infinite_keys_take_all_or_nothing(cuda_device, dtype, n):
    """A score of -inf leaves its key out, one of +inf leaves no finite output (inf - inf), and only in its head."""
    c = make(cuda_device, [n, 77], 8, 2, 64, 16, dtype, seed=n + 1)
    pg, row = at(c, 0, 7)
    c["k"][pg, row, 0] = 0
    c["q"][0, :4, 5] = torch.tensor([1.0, -1.0, -2.0, 0.5], device=cuda_device, dtype=dtype)
    plain, _ = run(c)
    c["k"][pg, row, 0, 5] = math.inf
    got, lse = run(c)
    up, down = [0, 3], [1, 2]
    assert not bool(torch.isfinite(got[0, up]).any()) and not bool(torch.isfinite(lse[0, up]).any())
    assert torch.equal(got[0, 4:], plain[0, 4:]) and torch.equal(got[1], plain[1])
    c["k"][pg, row, 0, 5] = 30000.0 if dtype == HF else 1e30      # far below every other score
    left_out, _ = run(c)
    assert torch.equal(got[0, down], left_out[0, down])


@pytest.mark.parametrize("cache", [BF, HF, E4])
def test_nan_keys_and_queries_show_in_their_heads(cuda_device, cache):
    c = make(cuda_device, [900, 77], 8, 2, 64, 16, cache if cache != E4 else BF, cache, seed=3)
    want, _ = run(c)
    pg, row = at(c, 0, 500)
    old = c["k"][pg, row, 1, 2].clone()
    c["k"][pg, row, 1, 2] = math.nan
    got, lse = run(c)
    assert bool(torch.isnan(got[0, 4:]).all()) and bool(torch.isnan(lse[0, 4:]).all())
    assert torch.equal(got[0, :4], want[0, :4]) and torch.equal(got[1], want[1])
    c["k"][pg, row, 1, 2] = old
    c["q"][1, 6, 63] = math.nan
    got, _ = run(c)
    assert bool(torch.isnan(got[1, 6]).all())
    keep = [h for h in range(8) if h != 6]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1, keep], want[1, keep])
