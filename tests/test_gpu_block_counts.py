"""The largest row counts that the block's entry points take (2^31 - 1): row numbers and grids at the end of 32 bits."""
import pytest
import torch

import mixture_experts_decode_gb300 as moe

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0
    torch.cuda.empty_cache()


def test_rope_of_the_most_tokens(cuda_device):
    """Every token has the same heads of one element (strides 0); the last token alone has a slot."""
    q = torch.full((1, 1, 1), 3.0, dtype=BF, device=cuda_device).expand(MOST, 1, 1)
    k = torch.full((1, 1, 1), 5.0, dtype=BF, device=cuda_device).expand(MOST, 1, 1)
    cache = torch.zeros(2, 8, 1, 1, dtype=BF, device=cuda_device)
    values = torch.zeros_like(cache)
    pos = torch.zeros(MOST, dtype=torch.int32, device=cuda_device)
    slots = torch.full((MOST,), -1, dtype=torch.int64, device=cuda_device)
    slots[-1] = 11
    out = torch.zeros(MOST + 64, dtype=BF, device=cuda_device)
    moe.rope_append(q, k, q, pos, slots, torch.empty(0, dtype=torch.float64, device=cuda_device), cache, values,
                    q_out=out[32:32 + MOST].view(MOST, 1, 1))
    torch.cuda.synchronize()
    assert bool((out[32:32 + MOST] == 3).all()) and not bool(out[:32].any()) and not bool(out[32 + MOST:].any())
    want = torch.zeros(16, device=cuda_device)
    want[11] = 1
    assert torch.equal(cache.view(-1).float(), 5 * want) and torch.equal(values.view(-1).float(), 3 * want)


def test_norm_of_the_most_rows(cuda_device):
    """d = 1, four rows a block; RMS norm makes each row its sign."""
    y = torch.ones(MOST, dtype=BF, device=cuda_device)
    y[-1] = -2
    y[MOST // 2] = -3
    out = torch.zeros(MOST + 64, dtype=BF, device=cuda_device)
    moe.norm_residual(y.view(MOST, 1), pre=moe.Norm(eps=0.0), out=out[32:32 + MOST].view(MOST, 1))
    torch.cuda.synchronize()
    assert float(out[32 + MOST - 1]) == -1 and float(out[32 + MOST // 2]) == -1
    assert int((out[32:32 + MOST] == 1).sum()) == MOST - 2
    assert not bool(out[:32].any()) and not bool(out[32 + MOST:].any())


@pytest.mark.parametrize("T", [1, 2])
def test_matvec_of_the_most_weight_rows(cuda_device, T):
    """K = 32 (34 GB of codes): weight rows of 8 - 8 = 0 except the first, a middle and the last one."""
    free, _ = torch.cuda.mem_get_info()
    if free < 80 << 30:
        pytest.skip("needs 80 GB free")
    codes = torch.full((MOST, 16), 0x88, dtype=torch.uint8, device=cuda_device)
    scales = torch.ones(MOST, 1, dtype=HF, device=cuda_device)
    rows = {0: 1, MOST // 2: 2, MOST - 1: 3}
    for r, w in rows.items():
        codes[r] = (8 + w) * 0x11
    x = torch.full((T, 32), 0.5, dtype=HF, device=cuda_device)
    y = moe.matvec4(x, moe.W4(codes, scales))
    torch.cuda.synchronize()
    for t in range(T):
        for r, w in rows.items():
            assert float(y[t, r]) == 16 * w
        assert int((y[t] != 0).sum()) == len(rows)
