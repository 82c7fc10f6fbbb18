// block_common.cuh -- device helpers of the kernels around the expert layer.
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

// Types of a key-value cache.
constexpr int KV_BF16 = 0, KV_F16 = 1, KV_E4M3 = 2;

// Two floats as 16-bit values of a word, lo in the lower half.
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (BF)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two E4M3 codes in the low / high half of a word -> FP16 pair, exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{ .reg .b16 l, h;\n\t mov.b32 {l, h}, %2;\n\t cvt.rn.f16x2.e4m3x2 %0, l;\n\t cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// 2^x within 2 units in the last place; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_ftz(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The reference of weights whose scores are all -inf is 0.
__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.f : m; }

// The warp's index in its block as a value the compiler knows to be the same
// in all lanes: branches on it do not split the warp.
__device__ __forceinline__ int warp_index() { return __shfl_sync(FULL_MASK, (int)threadIdx.x >> 5, 0); }

// The kernels of the decode block are launched as programmatic dependents:
// their blocks may be set up while the kernel before them in the stream ends,
// and each begins with after_previous(), which waits until that kernel has
// completed and its writes are visible.  (Two begin earlier, behind a kernel
// that has itself waited and lets them: the shared prefix's and the page plan's
// second launch.  They read past L1 and wait at their end.)  A step is a chain of kernels of a few
// microseconds; this takes about 2 us off the gap between two calls (attention
// of 777 keys in a loop of calls 12.4 -> 9.9 us, 4-bit 16 x 4096 -> 7169 14.4
// -> 12.3 us).  A block of such a kernel may be resident while its inputs are
// still being written, so they are not read-only for the kernel's duration and
// are read by ordinary loads, never through the non-coherent path
// (ld.global.nc, __ldg): the wait orders the writes before the former only.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The kernel behind this one in the stream may be set up from here on (once
// every block has come here), not only from this one's end on.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
