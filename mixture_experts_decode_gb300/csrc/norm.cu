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
// Bound: HBM, every operand in or out once; for one row, latency.  One to
// sixteen warps hold a row, as NV vectors of VW elements per thread: VW is 8,
// or what d and the addresses allow (4, 1).  The residual and the gate are
// loaded as they lie before the first reduction, and kept unconverted until
// used, so that two blocks of 512 threads fit an SM and one's loads run under
// the other's reductions.  Rows beyond 16384 go through shared memory.
// Measured: 8192 rows of 7168, both norms, sigmoid gate, FP32 residual (822
// MB): 140 us, 5.9 TB/s; one row of 2048: 1.9 us.
#include <algorithm>

#include "block_common.cuh"
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
template <bool BF>
__device__ __forceinline__ float2 norm_to_f2(uint32_t w) {
    if (BF) return bf16x2_to_float2(w);
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}
template <bool BF>
__device__ __forceinline__ uint32_t norm_from_f2(float a, float b) {
    uint32_t r;
    if (BF)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// VW consecutive elements as they lie in memory: 16-bit (F32 false) or 32-bit.
template <int VW, bool F32>
struct Raw {
    uint32_t w[F32 ? VW : (VW + 1) / 2];
};
template <int VW, bool F32>
__device__ __forceinline__ Raw<VW, F32> raw_load(const void* p, int64_t at) {
    Raw<VW, F32> r;
    if constexpr (F32) {
        const float* q = static_cast<const float*>(p) + at;
        if constexpr (VW >= 4) {
#pragma unroll
            for (int i = 0; i < VW / 4; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(q)[i];
                r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
            }
        } else {
            r.w[0] = __float_as_uint(q[0]);
        }
    } else {
        const uint16_t* q = static_cast<const uint16_t*>(p) + at;
        if constexpr (VW == 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(q);
            r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
        } else if constexpr (VW == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(q);
            r.w[0] = v.x, r.w[1] = v.y;
        } else {
            r.w[0] = q[0];
        }
    }
    return r;
}
template <int VW, bool BF, bool F32>
__device__ __forceinline__ void raw_floats(const Raw<VW, F32>& r, float (&f)[VW]) {
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < VW; ++j) f[j] = __uint_as_float(r.w[j]);
    } else if constexpr (VW == 1) {
        f[0] = norm_to_f<BF>((uint16_t)r.w[0]);
    } else {
#pragma unroll
        for (int j = 0; j < VW / 2; ++j) {
            const float2 v = norm_to_f2<BF>(r.w[j]);
            f[2 * j] = v.x, f[2 * j + 1] = v.y;
        }
    }
}
template <int VW, bool BF, bool F32>
__device__ __forceinline__ void raw_store(void* p, int64_t at, const float (&f)[VW]) {
    if constexpr (F32) {
        float* q = static_cast<float*>(p) + at;
        if constexpr (VW >= 4) {
#pragma unroll
            for (int i = 0; i < VW / 4; ++i)
                reinterpret_cast<float4*>(q)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        } else {
            q[0] = f[0];
        }
    } else {
        uint16_t* q = static_cast<uint16_t*>(p) + at;
        if constexpr (VW == 8)
            *reinterpret_cast<uint4*>(q) = make_uint4(norm_from_f2<BF>(f[0], f[1]), norm_from_f2<BF>(f[2], f[3]),
                                                      norm_from_f2<BF>(f[4], f[5]), norm_from_f2<BF>(f[6], f[7]));
        else if constexpr (VW == 4)
            *reinterpret_cast<uint2*>(q) = make_uint2(norm_from_f2<BF>(f[0], f[1]), norm_from_f2<BF>(f[2], f[3]));
        else
            q[0] = norm_from_f<BF>(f[0]);
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
// (the fast exponential and reciprocal are off by a few units of 2^-22 for
// gates of ordinary size, far below any output's rounding)
__device__ __forceinline__ float gate_value(float g, int act) {
    return act == MOE_GATE_SIGMOID ? __fdividef(1.f, 1.f + __expf(-g)) : g;
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
    for (int o = WARPS / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    v = __shfl_sync(FULL_MASK, v, 0);
    phase ^= 1;
    return v;
}

// The norm of a row held as NV vectors per thread (zeros beyond d).
template <int WARPS, int NV, int VW, bool BF>
__device__ __forceinline__ void norm_row(float (&f)[NV][VW], const NormSpec& s, int d, int first,
                                         float (*scratch)[32], int& phase) {
    constexpr int stride = WARPS * 32;
    if (s.kind == MOE_NORM_LAYER) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VW; ++j) sum += f[i][j];
        const float mean = row_sum<WARPS>(sum, scratch, phase) / d;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((first + i * stride) * VW < d)
#pragma unroll
                for (int j = 0; j < VW; ++j) f[i][j] -= mean;
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VW; ++j) sq += f[i][j] * f[i][j];
    const float inv = 1.f / sqrtf(row_sum<WARPS>(sq, scratch, phase) / d + s.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (first + i * stride) * VW;
        if (at < d) {
#pragma unroll
            for (int j = 0; j < VW; ++j) f[i][j] *= inv;
            float w[VW];
            if (s.w) {
                raw_floats<VW, BF, false>(raw_load<VW, false>(s.w, at), w);
#pragma unroll
                for (int j = 0; j < VW; ++j) f[i][j] *= w[j];
            }
            if (s.b) {
                raw_floats<VW, BF, false>(raw_load<VW, false>(s.b, at), w);
#pragma unroll
                for (int j = 0; j < VW; ++j) f[i][j] += w[j];
            }
        }
    }
}

}  // namespace

// Blocks per SM that the registers are cut for: as many as do not spill.
constexpr int norm_min_blocks(int warps, int nv, int vw) {
    const bool heavy = nv * vw > 16 || nv >= 16;
    return warps == 16 ? (heavy ? 1 : 2) : warps == 8 ? 4 : heavy ? 4 : 8;
}

// WARPS warps hold a row, NV vectors of VW elements per thread (WARPS = 1:
// four rows per block, one per warp).
template <int WARPS, int NV, int VW, bool BF, bool RF>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : WARPS * 32, norm_min_blocks(WARPS, NV, VW))
    norm_rows_kernel(const NormArgs a) {
    __shared__ float scratch[2][32];
    after_previous();
    const int64_t row = WARPS == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.T) return;  // (WARPS = 1 has no barriers)
    const int first = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
    constexpr int stride = WARPS * 32;
    const bool gate_full = a.gate && a.gate_col;
    int phase = 0;
    float f[NV][VW];
    Raw<VW, RF> r[NV];
    Raw<VW, false> gt[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (first + i * stride) * VW;
        if (at < a.d) {
            raw_floats<VW, BF, false>(raw_load<VW, false>(a.y, row * a.y_stride + at), f[i]);
            if (a.resid) r[i] = raw_load<VW, RF>(a.resid, row * a.r_stride + at);
            if (gate_full) gt[i] = raw_load<VW, false>(a.gate, row * a.gate_row + at);
        } else {
#pragma unroll
            for (int j = 0; j < VW; ++j) f[i][j] = 0.f;
        }
    }
    const float scale = a.alpha * (a.gate && !gate_full
                                       ? gate_value(row_load<BF, false>(a.gate, row * a.gate_row), a.gate_act) : 1.f);
    if (a.post.kind >= 0) norm_row<WARPS, NV, VW, BF>(f, a.post, a.d, first, scratch, phase);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (first + i * stride) * VW;
        if (at < a.d) {
            if (gate_full) {
                float g[VW];
                raw_floats<VW, BF, false>(gt[i], g);
                if (a.gate_act == MOE_GATE_SIGMOID) {
#pragma unroll
                    for (int j = 0; j < VW; ++j) g[j] = gate_value(g[j], MOE_GATE_SIGMOID);
                }
#pragma unroll
                for (int j = 0; j < VW; ++j) f[i][j] *= g[j];
            }
            if (a.resid) {
                float v[VW];
                raw_floats<VW, BF, RF>(r[i], v);
#pragma unroll
                for (int j = 0; j < VW; ++j) f[i][j] = v[j] + scale * f[i][j];
            } else {
#pragma unroll
                for (int j = 0; j < VW; ++j) f[i][j] *= scale;
            }
            if (a.resid_out) raw_store<VW, BF, RF>(a.resid_out, row * a.d + at, f[i]);
        }
    }
    if (!a.out) return;
    if (a.pre.kind >= 0) norm_row<WARPS, NV, VW, BF>(f, a.pre, a.d, first, scratch, phase);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (first + i * stride) * VW;
        if (at < a.d) raw_store<VW, BF, false>(a.out, row * a.d + at, f[i]);
    }
}

// Any length and alignment: the row as FP32 in shared memory.
constexpr int NORM_ANY_WARPS = 16;
template <bool BF, bool RF>
__global__ void __launch_bounds__(NORM_ANY_WARPS * 32) norm_any_kernel(const NormArgs a) {
    extern __shared__ float sm_row[];
    __shared__ float scratch[2][32];
    constexpr int TH = NORM_ANY_WARPS * 32;
    after_previous();
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

template <int WARPS, int NV, int VW, bool BF, bool RF>
static cudaError_t norm_rows(const NormArgs& a, cudaStream_t st) {
    constexpr int rows = WARPS == 1 ? 4 : 1;
    return launch_after(norm_rows_kernel<WARPS, NV, VW, BF, RF>, dim3((a.T - 1) / rows + 1), WARPS == 1 ? 128 : WARPS * 32, 0,
                        st, a);
}

template <bool BF, bool RF>
static cudaError_t launch_norm(const NormArgs& a, const DeviceInfo& di, cudaStream_t st) {
    // the widest vector that d and every address allow
    auto fits = [&](int vw) {
        auto al = [&](const void* p, int64_t stride, int es) {
            return reinterpret_cast<uintptr_t>(p) % std::min(vw * es, 16) == 0 && stride % vw == 0;
        };
        const int rs = RF ? 4 : 2;
        return a.d % vw == 0 && al(a.y, a.y_stride, 2) && al(a.resid, a.r_stride, rs) &&
               (a.gate_col == 0 || al(a.gate, a.gate_row, 2)) && al(a.post.w, 0, 2) && al(a.post.b, 0, 2) &&
               al(a.pre.w, 0, 2) && al(a.pre.b, 0, 2) && al(a.resid_out, 0, rs) && al(a.out, 0, 2);
    };
    // a warp per row once the rows fill the GPU's warps; several for fewer rows, for latency
    const bool many = a.T >= di.sm_count * 8;
    if (a.d > 16384) {
        static SmemOnce once;
        const cudaError_t e = once.set(reinterpret_cast<const void*>(norm_any_kernel<BF, RF>), MOE_NORM_MAX_DIM * 4);
        if (e != cudaSuccess) return e;
        return launch_after(norm_any_kernel<BF, RF>, dim3(a.T), NORM_ANY_WARPS * 32, (size_t)a.d * 4, st, a);
    }
    if (fits(8)) {
        if (a.d <= 128) return norm_rows<1, 1, 4, BF, RF>(a, st);
        if (a.d <= 256) return norm_rows<1, 1, 8, BF, RF>(a, st);
        if (a.d <= 512 && many) return norm_rows<1, 2, 8, BF, RF>(a, st);
        if (a.d <= 1024 && many) return norm_rows<1, 4, 8, BF, RF>(a, st);
        if (a.d <= 1024) return norm_rows<4, 1, 8, BF, RF>(a, st);
        if (a.d <= 2048) return norm_rows<8, 1, 8, BF, RF>(a, st);
        if (a.d <= 4096) return norm_rows<16, 1, 8, BF, RF>(a, st);
        if (a.d <= 8192) return norm_rows<16, 2, 8, BF, RF>(a, st);
        return norm_rows<16, 4, 8, BF, RF>(a, st);
    }
    if (fits(4)) {
        if (a.d <= 128) return norm_rows<1, 1, 4, BF, RF>(a, st);
        if (a.d <= 256) return norm_rows<1, 2, 4, BF, RF>(a, st);
        if (a.d <= 512) return norm_rows<1, 4, 4, BF, RF>(a, st);
        if (a.d <= 2048) return norm_rows<4, 4, 4, BF, RF>(a, st);
        if (a.d <= 8192) return norm_rows<16, 4, 4, BF, RF>(a, st);
        return norm_rows<16, 8, 4, BF, RF>(a, st);
    }
    if (a.d <= 128) return norm_rows<1, 4, 1, BF, RF>(a, st);
    if (a.d <= 512) return norm_rows<4, 4, 1, BF, RF>(a, st);
    if (a.d <= 2048) return norm_rows<8, 8, 1, BF, RF>(a, st);
    if (a.d <= 4096) return norm_rows<16, 8, 1, BF, RF>(a, st);
    if (a.d <= 8192) return norm_rows<16, 16, 1, BF, RF>(a, st);
    return norm_rows<16, 32, 1, BF, RF>(a, st);
}

cudaError_t launch_norm_residual(const NormArgs& a, int dtype, int resid_dtype, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const bool rf = resid_dtype == MOE_F32;
    if (dtype == MOE_BF16) return rf ? launch_norm<true, true>(a, di, st) : launch_norm<true, false>(a, di, st);
    return rf ? launch_norm<false, true>(a, di, st) : launch_norm<false, false>(a, di, st);
}

}  // namespace moedec
