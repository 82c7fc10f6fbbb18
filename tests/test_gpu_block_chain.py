"""The block's kernels right behind the kernels that write their inputs, at the same addresses call after call
(each may be set up while the one before it still runs)."""
import pytest
import torch

import mixture_experts_decode_gb300 as moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("T,N", [(1, 2048), (1, 9984), (5, 2048), (16, 4096)])
def test_products_of_freshly_written_rows_and_weights(cuda_device, T, N):
    K, steps = 2048, 20
    g = torch.Generator(device=cuda_device).manual_seed(N + T)
    ys = torch.randn(steps, T, K, generator=g, device=cuda_device).to(BF)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=cuda_device, dtype=torch.uint8)
    scales = torch.rand(steps, N, K // 64, generator=g, device=cuda_device).to(BF)
    zeros = torch.randint(0, 16, (steps, N, K // 64), generator=g, device=cuda_device, dtype=torch.uint8)
    want = []
    for i in range(steps):
        x = moe.norm_residual(ys[i], pre=moe.Norm())
        torch.cuda.synchronize()
        want.append(moe.matvec4(x, moe.W4(codes, scales[i].clone(), zeros[i].clone())))
        torch.cuda.synchronize()
    x, s, z = torch.empty(T, K, dtype=BF, device=cuda_device), torch.empty_like(scales[0]), torch.empty_like(zeros[0])
    w = moe.W4(codes, s, z)
    out = torch.empty(steps, T, N, dtype=BF, device=cuda_device)
    for captured in (False, True):
        out.zero_()

        def chain():
            for i in range(steps):
                z.copy_(zeros[i])
                s.copy_(scales[i])
                moe.norm_residual(ys[i], pre=moe.Norm(), out=x)
                moe.matvec4(x, w, y=out[i])

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                chain()
            graph.replay()
        else:
            chain()
        torch.cuda.synchronize()
        for i in range(steps):
            assert torch.equal(out[i], want[i]), (captured, i)
    assert moe.device_error(cuda_device) == 0
