// block_common.cuh -- device helpers of the attention and 4-bit kernels.
#pragma once

#include "common.cuh"

namespace moedec {

// 16 bytes global -> shared, L2 only; src_bytes = 0 fills the destination with zeros.
__device__ __forceinline__ void cp_async_16_zfill(void* smem, const void* gmem, int src_bytes) {
    const uint32_t a = (uint32_t)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(a), "l"(gmem), "r"(src_bytes) : "memory");
}

// 16 bytes by an ordinary load.
__device__ __forceinline__ uint4 ld_128(const void* p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}

// The warp's index in its block as a value the compiler knows to be the same
// in all lanes: branches on it do not split the warp.
__device__ __forceinline__ int warp_index() { return __shfl_sync(FULL_MASK, (int)threadIdx.x >> 5, 0); }

// The kernels of the decode block are launched as programmatic dependents:
// their blocks may be set up while the kernel before them in the stream ends,
// and each begins with after_previous(), which waits until that kernel has
// completed and its writes are visible.  A step is a chain of kernels of a few
// microseconds; this takes about 2 us off the gap between two calls (attention
// of 777 keys in a loop of calls 12.4 -> 9.9 us, 4-bit 16 x 4096 -> 7169 14.4
// -> 12.3 us).  A block of such a kernel may be resident while its inputs are
// still being written, so they are not read-only for the kernel's duration and
// are read by ordinary loads, never through the non-coherent path
// (ld.global.nc, __ldg): the wait orders the writes before the former only.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace moedec
