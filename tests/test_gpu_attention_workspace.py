"""The counters of moe_paged_attention's workspace: all of them are left zero, and values that no call can have left
are reported, in the counters of the second level of joins as in those of the first."""
import pytest
import torch

import mixture_experts_decode_gb300 as moe
from test_gpu_attention import BF, check, make

pytestmark = pytest.mark.gpu
COUNTERS = 4096          # MOE_ATTN_COUNTER_BYTES
SECOND = 640 * 4         # a counter for each block before them


@pytest.mark.parametrize("Hq,Hkv,D,lens", [(8, 2, 64, [5000, 70]), (16, 1, 256, [9000]), (8, 1, 128, [40000]),
                                           (8, 4, 64, [300000, 1, 0, 777]), (4, 4, 64, [3000] * 7)])
def test_every_counter_is_left_zero(cuda_device, Hq, Hkv, D, lens):
    ws = moe.attention_workspace(Hq, Hkv, D, cuda_device)
    c = make(cuda_device, lens, Hq, Hkv, D, 64, BF, seed=D)
    for _ in range(2):
        moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], workspace=ws)
        torch.cuda.synchronize()
        assert int(ws[:COUNTERS].max()) == 0
    assert moe.device_error(cuda_device) == 0


def test_every_counter_is_left_zero_by_calls_of_different_shapes(cuda_device):
    ws = moe.attention_workspace(64, 1, 256, cuda_device)
    for Hq, Hkv, D, lens in ((8, 2, 64, [5000, 70]), (16, 1, 256, [9000]), (64, 4, 128, [33] * 40), (8, 2, 64, [12000])):
        check(make(cuda_device, lens, Hq, Hkv, D, 64, BF, seed=D), ws=ws, what="kept workspace")
        assert int(ws[:COUNTERS].max()) == 0
    assert moe.device_error(cuda_device) == 0


@pytest.mark.parametrize("dirty", [slice(0, SECOND), slice(SECOND, COUNTERS)])
def test_counters_beyond_any_call_are_reported(cuda_device, dirty):
    """(5000 keys: 27 pieces, joined by eights and then together)"""
    c = make(cuda_device, [5000], 8, 1, 64, 64, BF, seed=15)
    ws = moe.attention_workspace(8, 1, 64, cuda_device)
    ws[dirty] = 77
    moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], workspace=ws)
    assert moe.device_error(cuda_device) & 0x10
    ws[:COUNTERS].zero_()
    check(c, ws=ws, what="cleared")
    assert moe.device_error(cuda_device) == 0
