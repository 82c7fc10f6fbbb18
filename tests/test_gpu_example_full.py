"""The example's decoder block where a sequence has filled its pages."""
import os
import sys

import pytest
import torch

import mixture_experts_decode_gb300 as moe
from mixture_experts_decode_gb300 import inputs

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_block  # noqa: E402

pytestmark = pytest.mark.gpu


def test_full_sequence_is_reported_and_leaves_the_others(cuda_device):
    b = decode_block.DecodeBlock(inputs.TINY, 4, 2, 64, batch=2, capacity=32, page=16, device=cuda_device, group=64)
    b.lens.copy_(torch.tensor([5, 31], dtype=torch.int32))
    resid = torch.randn(2, inputs.TINY.d, device=cuda_device)
    b.step(resid)
    assert moe.device_error(cuda_device) == 0
    cache = b.k_cache.clone(), b.v_cache.clone()
    b.step(resid)                                    # the second sequence's 33rd token
    assert moe.device_error(cuda_device) & 0x8
    assert bool(torch.isfinite(resid).all())
    row = int(b.table[0, 0]), 6                      # the first one's seventh: the only row written
    for now, old in zip((b.k_cache, b.v_cache), cache):
        changed = (now != old).flatten(2).any(-1).nonzero().tolist()
        assert changed == [list(row)]
