"""GPU tests of moe_rope_append on prompts: many tokens a block, one after the other.

A call on a prompt must leave, bit for bit, what calls on slices of at most 256
tokens leave (there every block has one token, so no round of a block follows
another); beside that, the 64-bit reference and bounds of test_gpu_block_ops."""
import pytest
import torch

import mixture_experts_decode_gb300 as moe
from test_gpu_block_ops import rope_case, rope_check, raw

pytestmark = pytest.mark.gpu
BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0


def append(c, interleaved, lo=0, hi=None):
    cut = slice(lo, hi)
    return moe.rope_append(c["q"][cut], c["k"][cut], c["v"][cut], c["pos"][cut], c["slots"][cut], c["freqs"], c["kc"], c["vc"],
                           interleaved=interleaved, k_scale=c["ks"], v_scale=c["vs"])


def pad_some(c, seed):
    """About one token in nine without a slot."""
    g = torch.Generator(device=c["slots"].device).manual_seed(seed)
    c["slots"][torch.rand(c["slots"].shape, generator=g, device=c["slots"].device) < 1 / 9] = -1
    return c


@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [(16384, 32, 4, 128, 128), (16381, 32, 4, 128, 64), (20011, 2, 1, 64, 64),
                                            (9001, 8, 8, 80, 32), (5003, 5, 3, 256, 256), (7001, 4, 2, 128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("cache", [BF, E4])
def test_prompt_equals_its_slices(cuda_device, T, Hq, Hkv, D, rot, interleaved, cache):
    c = pad_some(rope_case(cuda_device, T, Hq, Hkv, D, rot, page=64, cache=cache, seed=T, max_pos=200000), T)
    start = raw(c["kc"]).clone(), raw(c["vc"]).clone()
    want_q = torch.cat([append(c, interleaved, t, t + 256) for t in range(0, T, 256)])
    want = raw(c["kc"]).clone(), raw(c["vc"]).clone()
    for _ in range(3):
        raw(c["kc"]).copy_(start[0])
        raw(c["vc"]).copy_(start[1])
        q = append(c, interleaved)
        assert torch.equal(raw(q), raw(want_q))
        assert torch.equal(raw(c["kc"]), want[0]) and torch.equal(raw(c["vc"]), want[1])


@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [(4999, 8, 2, 128, 128), (6007, 3, 1, 64, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("cache", [HF, E4])
def test_prompt_of_few_heads(cuda_device, T, Hq, Hkv, D, rot, interleaved, cache):
    rope_check(pad_some(rope_case(cuda_device, T, Hq, Hkv, D, rot, dtype=HF, cache=cache, seed=T), T), interleaved,
               what=f"T={T}")


# More heads than a block's threads have jobs for (four for each of 256 / units
# groups): heads are then taken one token at a time.  Head counts that no group
# count divides, whole and partial rotation, several tokens a block.
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved", [
    (1000, 61, 5, 256, 256, False), (1900, 71, 3, 128, 32, False), (700, 131, 7, 128, 128, False),
    (1, 67, 3, 128, 128, True), (2001, 67, 3, 128, 128, True), (1500, 129, 4, 64, 16, True), (900, 64, 8, 128, 64, True),
    (500, 127, 127, 128, 128, False)])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
def test_prompt_of_many_heads(cuda_device, T, Hq, Hkv, D, rot, interleaved, dtype, cache):
    c = pad_some(rope_case(cuda_device, T, Hq, Hkv, D, rot, dtype=dtype, cache=cache, seed=T + Hq), T)
    rope_check(c, interleaved, mscale=1.25, what=f"T={T} heads={Hq}/{Hkv}")
