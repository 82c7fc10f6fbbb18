"""The block's calls captured into graphs in the ways that programs capture: behind a copy or a clear, joined from two
streams, with a workspace made inside."""
import pytest
import torch

import mixture_experts_decode_gb300 as moe
from test_gpu_attention import BF, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    yield
    assert moe.device_error(cuda_device) == 0


def test_attention_with_its_workspace_made_inside(cuda_device):
    c = make(cuda_device, [2000, 300], 8, 2, 128, 64, BF, seed=1)
    call = lambda: moe.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"])  # noqa: E731
    want = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_calls_joined_from_two_streams(cuda_device):
    """Each call's inputs come from both streams, by kernels and by copies."""
    g = torch.Generator(device=cuda_device).manual_seed(2)
    d = 2048
    y, r = (torch.randn(4, d, generator=g, device=cuda_device).to(BF) for _ in range(2))
    w = moe.W4(torch.randint(0, 256, (d, d // 2), generator=g, device=cuda_device, dtype=torch.uint8),
               (torch.rand(d, d // 64, generator=g, device=cuda_device) * 0.01).to(BF))

    a, b, held = torch.empty_like(y), torch.empty_like(r), torch.empty_like(r)

    def body(side):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            held.copy_(r)
            moe.matvec4(held, w, y=b)
        a.copy_(y)
        moe.matvec4(a, w, y=a_out)
        main.wait_stream(side)
        return moe.norm_residual(a_out, b, pre=moe.Norm())

    a_out = torch.empty_like(y)
    want = moe.norm_residual(moe.matvec4(y, w), moe.matvec4(r, w), pre=moe.Norm())
    side = torch.cuda.Stream()
    got = body(side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, z) for x, z in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = body(side)
    for i in range(5):
        y.copy_(torch.randn(4, d, generator=g, device=cuda_device))
        r.copy_(torch.randn(4, d, generator=g, device=cuda_device))
        want = moe.norm_residual(moe.matvec4(y, w), moe.matvec4(r, w), pre=moe.Norm())
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, z) for x, z in zip(got, want)), i
