"""moe_matvec4 where the elements of x differ widely in size: what FP32 sums keep must be kept, whichever kernel takes
the call.  One row of x is split into 8-bit parts inside when the weight rows make two block tiles for every SM: from
N = 9697 where K is 2048 or more, 19393 at K = 1024, 77569 at K up to 256."""
import math

import pytest
import torch

import _block_refs as refs
import mixture_experts_decode_gb300 as moe
from test_gpu_block_ops import within

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0


def weights(dev, N, K, group, dtype, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    scales = torch.rand(N, K // group, generator=g, device=dev).to(dtype)
    zeros = torch.randint(0, 16, (N, K // group), generator=g, device=dev, dtype=torch.uint8)
    return codes, scales, zeros, g


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,N", [(1, 9984), (1, 130), (2, 9984)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_outlier_under_its_zero_point(cuda_device, dtype, T, N, group):
    """One large element whose weight is zero in every row, alone in its group: its products and its group's sum are
    exact in FP32 and cancel, so the bound is that of the other elements, far below it."""
    K, at = 2048, 257
    codes, scales, zeros, g = weights(cuda_device, N, K, group, dtype, group + N)
    zeros[:, at // group] = codes[:, at // 2] >> 4     # (an odd place is the high half of its byte)
    small = torch.randn(T, K, generator=g, device=cuda_device) * 2.0 ** -9
    lo = at // group * group
    small[:, lo:lo + group] = 0
    small = small.to(dtype)
    x = small.clone()
    x[:, at] = 2.0 ** 13
    want, bound = refs.matvec4(small, codes, scales, zeros, group)
    within(moe.matvec4(x, moe.W4(codes, scales, zeros)), want, bound, dtype, "outlier")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("N,K,group", [(9985, 2048, 64), (9985, 4224, 128), (19500, 1024, 32), (77600, 96, 32),
                                       (9985, 20000, 32)])
def test_one_row_of_wide_range(cuda_device, dtype, N, K, group):
    """Elements over 24 binades, and groups of very different size, within FP32's own bound."""
    codes, scales, zeros, g = weights(cuda_device, N, K, group, dtype, K)
    for spread in (1, 24):
        x = torch.randn(1, K, generator=g, device=cuda_device)
        by_group = 2.0 ** -torch.randint(0, spread, (1, K // group), generator=g, device=cuda_device).float()
        x = x * 2.0 ** -torch.randint(0, 25 - spread + 1, x.shape, generator=g, device=cuda_device).float()
        x = (x * by_group.repeat_interleave(group, 1)).to(dtype)
        want, bound = refs.matvec4(x, codes, scales, zeros, group)
        got = moe.matvec4(x, moe.W4(codes, scales, zeros))
        within(got, want, bound, dtype, f"spread {spread}")
        # a second row does not change the first one's bound
        got = moe.matvec4(torch.cat((x, -x)), moe.W4(codes, scales, zeros))
        within(got, torch.cat((want, -want)), torch.cat((bound, bound)), dtype, f"two rows, spread {spread}")


@pytest.mark.parametrize("dtype", [BF, HF])
def test_one_row_of_extreme_size(cuda_device, dtype):
    """Single elements at the ends of the type's range, each alone in its row: one product, rounded once."""
    K, N, group = 2048, 9984, 32
    codes, _, zeros, _ = weights(cuda_device, N, K, group, dtype, 1)
    tiny, most = torch.finfo(dtype).smallest_normal, torch.finfo(dtype).max
    for at, size, scale in ((0, tiny, 1.0), (33, -4 * tiny, 2.0), (2047, most / 2 ** 8, 2.0 ** -4), (64, -most / 2 ** 9, 0.5)):
        scales = torch.full((N, K // group), scale, dtype=dtype, device=cuda_device)
        x = torch.zeros(1, K, dtype=dtype, device=cuda_device)
        x[0, at] = size
        w = (codes[:, at // 2] >> (4 * (at % 2)) & 15).double() - zeros[:, at // group].double()
        got = moe.matvec4(x, moe.W4(codes, scales, zeros))
        assert torch.equal(got[0], (w * scale * x[0, at].double()).to(dtype)), (at, size)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,N", [(1, 9984), (1, 70), (3, 9984), (12, 300)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_infinities_show(cuda_device, dtype, T, N, bad):
    """No output of a row of x that holds an infinity or a NaN is finite; the other rows are as they were."""
    K, group = 2048, 64
    codes, scales, zeros, g = weights(cuda_device, N, K, group, dtype, 2)
    x = torch.randn(T, K, generator=g, device=cuda_device).to(dtype)
    clean = moe.matvec4(x, moe.W4(codes, scales, zeros))
    x[T // 2, 301] = bad
    got = moe.matvec4(x, moe.W4(codes, scales, zeros))
    assert not bool(torch.isfinite(got[T // 2]).any())
    keep = [t for t in range(T) if t != T // 2]
    assert torch.equal(got[keep], clean[keep])
