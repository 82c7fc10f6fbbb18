// norm.cu -- the step between two blocks of a decoder in one pass: the norm
// after a block, its gate, the scaled residual sum, and the norm before the
// next block.
//
// Mathematics, per row:
//   u = post(y),  r' = r + alpha * u * act(gate),  x = pre(r')
// with post / pre either absent, RMS  v / sqrt(mean(v^2) + eps) * w (+ b), or
// layer norm (the mean taken off first).  A row stays in registers as FP32
// from its load to its stores, so x is computed from the unrounded r' and each
// output is rounded once; a layer norm's variance is the mean of the centred
// squares (a second reduction), not a difference of moments.
//
// Bound: HBM, every operand in or out once.  A warp or a block holds a row
// (vectors of 8 elements, at most 4 per thread), so statistics cost one
// reduction in registers each; rows that are odd, unaligned or longer than
// 16384 go through a block with the row in shared memory.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moedec {

namespace {

template <bool BF>
__device__ __forceinline__ float norm_to_f(uint16_t v) {
    if (BF) return __uint_as_float((uint32_t)v << 16);
    __half h;
    memcpy(&h, &v, 2);
    return __half2float(h);
}
template <bool BF>
__device__ __forceinline__ uint16_t norm_from_f(float f) {
    uint16_t r;
    if (BF) {
        const __nv_bfloat16 v = __float2bfloat16_rn(f);
        memcpy(&r, &v, 2);
    } else {
        const __half v = __float2half_rn(f);
        memcpy(&r, &v, 2);
    }
    return r;
}

// Eight consecutive elements, 16-bit or (F32) 32-bit.
template <bool BF, bool F32>
__device__ __forceinline__ void row_load8(const void* p, int64_t at, float (&f)[8]) {
    if (F32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 a = q[0], b = q[1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = norm_to_f<BF>((uint16_t)w[i]);
            f[2 * i + 1] = norm_to_f<BF>((uint16_t)(w[i] >> 16));
        }
    }
}
template <bool BF, bool F32>
__device__ __forceinline__ void row_store8(void* p, int64_t at, const float (&f)[8]) {
    if (F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)norm_from_f<BF>(f[2 * i]) | (uint32_t)norm_from_f<BF>(f[2 * i + 1]) << 16;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <bool BF, bool F32>
__device__ __forceinline__ float row_load(const void* p, int64_t at) {
    return F32 ? static_cast<const float*>(p)[at] : norm_to_f<BF>(static_cast<const uint16_t*>(p)[at]);
}
template <bool BF, bool F32>
__device__ __forceinline__ void row_store(void* p, int64_t at, float f) {
    if (F32)
        static_cast<float*>(p)[at] = f;
    else
        static_cast<uint16_t*>(p)[at] = norm_from_f<BF>(f);
}
__device__ __forceinline__ float gate_value(float g, int act) {
    return act == MOE_GATE_SIGMOID ? 1.f / (1.f + expf(-g)) : g;
}

// Sum over the WARPS warps that hold a row; scratch[2][32] alternates so that
// one barrier per reduction is enough.
template <int WARPS>
__device__ __forceinline__ float row_sum(float v, float (*scratch)[32], int& phase) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    if (WARPS == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) scratch[phase][warp] = v;
    __syncthreads();
    v = lane < WARPS ? scratch[phase][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    phase ^= 1;
    return v;
}

// The norm of a row held as NV vectors per thread.
template <int WARPS, int NV, bool BF>
__device__ __forceinline__ void norm_row(float (&f)[NV][8], const NormSpec& s, int d, int first, int stride,
                                         float (*scratch)[32], int& phase) {
    float mean = 0.f;
    if (s.kind == MOE_NORM_LAYER) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += f[i][j];
        mean = row_sum<WARPS>(sum, scratch, phase) / d;
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((first + i * stride) * 8 < d)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[i][j] -= mean;
                sq += f[i][j] * f[i][j];
            }
    const float inv = 1.f / sqrtf(row_sum<WARPS>(sq, scratch, phase) / d + s.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (first + i * stride) * 8;
        if (at < d) {
            float w[8];
            if (s.w) row_load8<BF, false>(s.w, at, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] *= s.w ? inv * w[j] : inv;
            if (s.b) {
                row_load8<BF, false>(s.b, at, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] += w[j];
            }
        }
    }
}

}  // namespace

// WARPS warps hold a row, NV vectors per thread (WARPS = 1: four rows per
// block, one per warp).
template <int WARPS, int NV, bool BF, bool RF>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : WARPS * 32) norm_rows_kernel(const NormArgs a) {
    __shared__ float scratch[2][32];
    const int warp = threadIdx.x >> 5;
    const int row = WARPS == 1 ? blockIdx.x * 4 + warp : blockIdx.x;
    if (row >= a.T) return;  // (WARPS = 1 has no barriers)
    const int first = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
    constexpr int stride = WARPS * 32;
    int phase = 0;
    float f[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (first + i * stride) * 8;
        if (at < a.d)
            row_load8<BF, false>(a.y, row * a.y_stride + at, f[i]);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
    }
    // the residual and the gate are on their way while the first norm reduces
    float r[NV][8], gt[NV][8];
    const float row_gate = a.gate && a.gate_col == 0
                               ? gate_value(row_load<BF, false>(a.gate, row * a.gate_row), a.gate_act) : 1.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (first + i * stride) * 8;
        if (at < a.d && a.resid) row_load8<BF, RF>(a.resid, row * a.r_stride + at, r[i]);
        if (at < a.d && a.gate && a.gate_col) row_load8<BF, false>(a.gate, row * a.gate_row + at, gt[i]);
    }
    if (a.post.kind >= 0) norm_row<WARPS, NV, BF>(f, a.post, a.d, first, stride, scratch, phase);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (first + i * stride) * 8;
        if (at < a.d) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gv = a.gate && a.gate_col ? gate_value(gt[i][j], a.gate_act) : row_gate;
                const float u = a.alpha * (a.gate ? f[i][j] * gv : f[i][j]);
                f[i][j] = a.resid ? r[i][j] + u : u;
            }
            if (a.resid_out) row_store8<BF, RF>(a.resid_out, (int64_t)row * a.d + at, f[i]);
        }
    }
    if (!a.out) return;
    if (a.pre.kind >= 0) norm_row<WARPS, NV, BF>(f, a.pre, a.d, first, stride, scratch, phase);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (first + i * stride) * 8;
        if (at < a.d) row_store8<BF, false>(a.out, (int64_t)row * a.d + at, f[i]);
    }
}

// Any length and alignment: the row as FP32 in shared memory.
constexpr int NORM_ANY_WARPS = 16;
template <bool BF, bool RF>
__global__ void __launch_bounds__(NORM_ANY_WARPS * 32) norm_any_kernel(const NormArgs a) {
    extern __shared__ float sm_row[];
    __shared__ float scratch[2][32];
    constexpr int TH = NORM_ANY_WARPS * 32;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    int phase = 0;
    auto norm = [&](const NormSpec& s) {  // each thread revisits its own elements only
        float mean = 0.f;
        if (s.kind == MOE_NORM_LAYER) {
            float sum = 0.f;
            for (int i = tid; i < a.d; i += TH) sum += sm_row[i];
            mean = row_sum<NORM_ANY_WARPS>(sum, scratch, phase) / a.d;
        }
        float sq = 0.f;
        for (int i = tid; i < a.d; i += TH) {
            const float v = sm_row[i] - mean;
            sm_row[i] = v;
            sq += v * v;
        }
        const float inv = 1.f / sqrtf(row_sum<NORM_ANY_WARPS>(sq, scratch, phase) / a.d + s.eps);
        for (int i = tid; i < a.d; i += TH) {
            float v = sm_row[i] * (s.w ? inv * row_load<BF, false>(s.w, i) : inv);
            if (s.b) v += row_load<BF, false>(s.b, i);
            sm_row[i] = v;
        }
    };
    for (int i = tid; i < a.d; i += TH) sm_row[i] = row_load<BF, false>(a.y, row * a.y_stride + i);
    if (a.post.kind >= 0) norm(a.post);
    for (int i = tid; i < a.d; i += TH) {
        float u = sm_row[i];
        if (a.gate) u *= gate_value(row_load<BF, false>(a.gate, row * a.gate_row + i * a.gate_col), a.gate_act);
        u *= a.alpha;
        const float v = a.resid ? row_load<BF, RF>(a.resid, row * a.r_stride + i) + u : u;
        sm_row[i] = v;
        if (a.resid_out) row_store<BF, RF>(a.resid_out, row * a.d + i, v);
    }
    if (!a.out) return;
    if (a.pre.kind >= 0) norm(a.pre);
    for (int i = tid; i < a.d; i += TH) row_store<BF, false>(a.out, row * a.d + i, sm_row[i]);
}

template <bool BF, bool RF>
static cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
    auto al = [](const void* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0; };
    const bool vec = a.d % 8 == 0 && a.d <= 16384 && al(a.y, a.y_stride) && al(a.resid, a.r_stride) &&
                     (a.gate_col == 0 || al(a.gate, a.gate_row)) && al(a.post.w, 0) && al(a.post.b, 0) &&
                     al(a.pre.w, 0) && al(a.pre.b, 0) && al(a.resid_out, 0) && al(a.out, 0);
    if (!vec) {
        static SmemOnce once;
        const cudaError_t e = once.set(reinterpret_cast<const void*>(norm_any_kernel<BF, RF>), MOE_NORM_MAX_DIM * 4);
        if (e != cudaSuccess) return e;
        norm_any_kernel<BF, RF><<<a.T, NORM_ANY_WARPS * 32, (size_t)a.d * 4, st>>>(a);
    } else if (a.d <= 256) {
        norm_rows_kernel<1, 1, BF, RF><<<(a.T + 3) / 4, 128, 0, st>>>(a);
    } else if (a.d <= 2048) {
        norm_rows_kernel<8, 1, BF, RF><<<a.T, 256, 0, st>>>(a);
    } else if (a.d <= 4096) {
        norm_rows_kernel<16, 1, BF, RF><<<a.T, 512, 0, st>>>(a);
    } else if (a.d <= 8192) {
        norm_rows_kernel<16, 2, BF, RF><<<a.T, 512, 0, st>>>(a);
    } else {
        norm_rows_kernel<16, 4, BF, RF><<<a.T, 512, 0, st>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_norm_residual(const NormArgs& a, int dtype, int resid_dtype, cudaStream_t st) {
    const bool rf = resid_dtype == MOE_F32;
    if (dtype == MOE_BF16) return rf ? launch_norm<true, true>(a, st) : launch_norm<true, false>(a, st);
    return rf ? launch_norm<false, true>(a, st) : launch_norm<false, false>(a, st);
}

}  // namespace moedec
