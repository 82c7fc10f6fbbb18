// block_common.cuh -- device helpers of the attention and 4-bit kernels.
#pragma once

#include "common.cuh"

namespace moedec {

// 16 bytes global -> shared, L2 only; src_bytes = 0 fills the destination with zeros.
__device__ __forceinline__ void cp_async_16_zfill(void* smem, const void* gmem, int src_bytes) {
    const uint32_t a = (uint32_t)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(a), "l"(gmem), "r"(src_bytes) : "memory");
}

// The warp's index in its block as a value the compiler knows to be the same
// in all lanes: branches on it do not split the warp.
__device__ __forceinline__ int warp_index() { return __shfl_sync(FULL_MASK, (int)threadIdx.x >> 5, 0); }

}  // namespace moedec
