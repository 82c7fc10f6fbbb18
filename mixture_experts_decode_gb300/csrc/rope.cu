// rope.cu -- rotary positions on the query and key heads of new tokens,
// fused with writing the rotated keys and the values into a paged cache.
//
// Mathematics.  Pair i of a head's first `rot` dims is (x_i, x_{i+rot/2}) in
// the half layout and (x_{2i}, x_{2i+1}) interleaved; with a = pos * f_i,
//   (x, y) -> mscale * (x cos a - y sin a,  y cos a + x sin a).
// The angle is reduced exactly: f_i / 2 pi is taken modulo 1 as a 64-bit
// fraction F_i of a turn (FP64, once per thread), and pos * F_i wraps modulo
// 2^64, that is modulo a whole turn, so a position of 2^31 still has its angle
// to 2^-34 turns, where an FP32 product would be off by radians.  The top 32
// bits, as a signed fraction of half a turn, go to sincospif.
//
// Bound: HBM, each element in and out once.  One block takes one token at a
// time (blocks stride over the tokens): its rot/2 sines go to shared memory
// once and serve every head.  All arithmetic is FP32; each output is rounded
// once (E4M3: divided by the cache's scale, nearest even, saturated at 448).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moedec {

namespace {

constexpr int ROPE_THREADS = 256;

template <bool BF>
__device__ __forceinline__ float to_f(uint16_t v) {
    if (BF) return __uint_as_float((uint32_t)v << 16);
    __half h;
    memcpy(&h, &v, 2);
    return __half2float(h);
}
template <bool BF>
__device__ __forceinline__ uint16_t from_f(float f) {
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
// Two floats -> two E4M3 codes (a in the low byte), nearest even, saturated.
__device__ __forceinline__ uint16_t e4m3_pair(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

template <bool BF>
__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = to_f<BF>((uint16_t)w[i]);
        f[2 * i + 1] = to_f<BF>((uint16_t)(w[i] >> 16));
    }
}
template <bool BF>
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)from_f<BF>(f[2 * i]) | (uint32_t)from_f<BF>(f[2 * i + 1]) << 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&f)[8], float scale) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = (uint32_t)e4m3_pair(f[4 * i] / scale, f[4 * i + 1] / scale) |
               (uint32_t)e4m3_pair(f[4 * i + 2] / scale, f[4 * i + 3] / scale) << 16;
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

}  // namespace

// One head's destination: query output rows, or cache rows (null: not written).
template <bool BF, bool E4>
struct RopeDst {
    uint8_t* p;  // E4 && cache: bytes; else 16-bit elements
    bool cache;
    float scale;
    __device__ __forceinline__ void put8(int dim, const float (&f)[8]) const {
        if (!p) return;
        if (E4 && cache)
            store8_e4m3(p + dim, f, scale);
        else
            store8<BF>(reinterpret_cast<uint16_t*>(p) + dim, f);
    }
    __device__ __forceinline__ void put(int dim, float f) const {
        if (!p) return;
        if (E4 && cache)
            p[dim] = (uint8_t)e4m3_pair(f / scale, 0.f);
        else
            reinterpret_cast<uint16_t*>(p)[dim] = from_f<BF>(f);
    }
};

// VEC: rows 16-byte aligned, D and the rotated halves (or pairs) in whole
// vectors of 8; otherwise one element (or pair) per thread.
template <bool BF, bool E4, bool VEC>
__global__ void __launch_bounds__(ROPE_THREADS) rope_append_kernel(const RopeArgs a) {
    __shared__ float2 sm_cs[2][ROPE_THREADS];  // cos, sin of the token's pairs
    __shared__ int64_t sm_slot[2][2];          // page (or -1), row within it
    constexpr int CES = E4 ? 1 : 2;
    const int tid = threadIdx.x;
    const int half = a.rot / 2;
    uint64_t F = 0;
    if (tid < half) {
        double turns = a.freqs[tid] * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= floor(turns);
        F = (uint64_t)(turns * 18446744073709551616.0);
    }
    const int inter = a.interleaved;
    // units of work of a rotated head, and of a value head
    const int rot_units = VEC ? (inter ? a.rot / 8 : a.rot / 16) : half;
    const int head_units = rot_units + (a.D - a.rot) / (VEC ? 8 : 1);
    const int v_units = a.D / (VEC ? 8 : 1);
    const int rot_total = (a.Hq + a.Hkv) * head_units;
    const int total = rot_total + a.Hkv * v_units;
    int buf = 0;
    for (int tok = blockIdx.x; tok < a.T; tok += gridDim.x, buf ^= 1) {
        if (tid < half) {
            const uint64_t phase = (uint64_t)(int64_t)a.positions[tok] * F;
            const float x = (float)(int32_t)(phase >> 32) * 4.656612873077393e-10f;  // 2^-31: half turns
            float s, c;
            sincospif(x, &s, &c);
            sm_cs[buf][tid] = make_float2(c * a.mscale, s * a.mscale);
        }
        if (tid == ROPE_THREADS - 1) {
            const int64_t slot = a.slots[tok];
            int64_t page = -1, row = 0;
            if (slot >= 0) {
                page = slot / a.page;
                row = slot - page * a.page;
                if (page >= a.num_pages) {
                    page = -1;
                    atomicOr(a.err, MOE_DEVERR_PAGE);
                }
            }
            sm_slot[buf][0] = page;
            sm_slot[buf][1] = row;
        }
        __syncthreads();  // (the other buffer's readers are past: one token apart)
        const int64_t page = sm_slot[buf][0], row = sm_slot[buf][1];
        for (int i = tid; i < total; i += ROPE_THREADS) {
            RopeDst<BF, E4> dst;
            const uint16_t* src;
            int unit;
            if (i < rot_total) {
                int h = i / head_units;
                unit = i - h * head_units;
                if (h < a.Hq) {
                    src = static_cast<const uint16_t*>(a.q) + tok * a.q_st + h * a.q_sh;
                    dst = {static_cast<uint8_t*>(a.q_out) + (tok * a.qo_st + h * a.qo_sh) * 2, false, 1.f};
                } else {
                    h -= a.Hq;
                    src = static_cast<const uint16_t*>(a.k) + tok * a.k_st + h * a.k_sh;
                    dst = {page < 0 ? nullptr
                                    : static_cast<uint8_t*>(a.kc) + (page * a.kc_sp + row * a.kc_st + h * a.kc_sh) * CES,
                           true, a.k_scale};
                }
            } else {
                const int j = i - rot_total;
                const int h = j / v_units;
                unit = j - h * v_units;
                src = static_cast<const uint16_t*>(a.v) + tok * a.v_st + h * a.v_sh;
                dst = {page < 0 ? nullptr
                                : static_cast<uint8_t*>(a.vc) + (page * a.vc_sp + row * a.vc_st + h * a.vc_sh) * CES,
                       true, a.v_scale};
            }
            const bool turn = i < rot_total && unit < rot_units;
            if (VEC) {
                const int dim = turn ? unit * 8 : (i < rot_total ? a.rot + (unit - rot_units) * 8 : unit * 8);
                float f[8];
                load8<BF>(src + dim, f);
                if (turn && inter) {
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float2 cs = sm_cs[buf][unit * 4 + p];
                        const float x = f[2 * p], y = f[2 * p + 1];
                        f[2 * p] = x * cs.x - y * cs.y;
                        f[2 * p + 1] = y * cs.x + x * cs.y;
                    }
                } else if (turn) {
                    float e[8];
                    load8<BF>(src + dim + half, e);
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        const float2 cs = sm_cs[buf][dim + p];
                        const float x = f[p], y = e[p];
                        f[p] = x * cs.x - y * cs.y;
                        e[p] = y * cs.x + x * cs.y;
                    }
                    dst.put8(dim + half, e);
                }
                dst.put8(dim, f);
            } else if (turn) {
                const int d0 = inter ? 2 * unit : unit, d1 = inter ? d0 + 1 : unit + half;
                const float2 cs = sm_cs[buf][unit];
                const float x = to_f<BF>(src[d0]), y = to_f<BF>(src[d1]);
                dst.put(d0, x * cs.x - y * cs.y);
                dst.put(d1, y * cs.x + x * cs.y);
            } else {
                const int dim = i < rot_total ? a.rot + unit - rot_units : unit;
                dst.put(dim, to_f<BF>(src[dim]));
            }
        }
    }
}

template <bool BF, bool E4>
static cudaError_t launch_rope(const RopeArgs& a, const DeviceInfo& di, cudaStream_t st) {
    const int grid = std::min(a.T, di.sm_count * 8);
    auto al = [](const void* p, int64_t s0, int64_t s1, int64_t s2) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 % 8 == 0 && s1 % 8 == 0 && s2 % 8 == 0;
    };
    const bool vec = a.D % 8 == 0 && a.rot % (a.interleaved ? 8 : 16) == 0 && al(a.q, a.q_st, a.q_sh, 0) &&
                     al(a.k, a.k_st, a.k_sh, 0) && al(a.v, a.v_st, a.v_sh, 0) && al(a.q_out, a.qo_st, a.qo_sh, 0) &&
                     al(a.kc, a.kc_sp, a.kc_st, a.kc_sh) && al(a.vc, a.vc_sp, a.vc_st, a.vc_sh);
    if (vec)
        rope_append_kernel<BF, E4, true><<<grid, ROPE_THREADS, 0, st>>>(a);
    else
        rope_append_kernel<BF, E4, false><<<grid, ROPE_THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_rope_append(RopeArgs a, int dtype, int cache_dtype, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    a.err = di.err_word;
    if (cache_dtype == MOE_E4M3) return dtype == MOE_BF16 ? launch_rope<true, true>(a, di, st) : launch_rope<false, true>(a, di, st);
    return dtype == MOE_BF16 ? launch_rope<true, false>(a, di, st) : launch_rope<false, false>(a, di, st);
}

}  // namespace moedec
