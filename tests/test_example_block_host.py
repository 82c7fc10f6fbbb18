"""The decode block example's slots of new tokens (no GPU)."""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_block  # noqa: E402


def test_slots_of_next_tokens_and_of_full_sequences():
    table = torch.tensor([[4, 1], [0, 3], [2, 5], [6, 7]], dtype=torch.int32)
    positions = torch.tensor([0, 17, 31, 32], dtype=torch.int32)
    first = decode_block.first_slots(table, 16, 8)
    slots = decode_block.cache_slots(first, positions, 16)
    assert slots.dtype == torch.int64
    assert slots.tolist() == [4 * 16, 3 * 16 + 1, 5 * 16 + 15, 8 * 16]   # the last one is past the cache
    assert decode_block.cache_slots(first, positions + 1024, 16).tolist() == [128, 129, 143, 128]
