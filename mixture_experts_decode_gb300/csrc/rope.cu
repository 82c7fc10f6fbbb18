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
// once and serve every head.  A thread keeps one place within a head (a
// 16-byte vector, or the two vectors of eight rotated pairs) for all the heads
// it visits, so that its sines sit in registers and the addresses of a head
// cost one multiplication; the first heads' loads are on their way before the
// sines are ready.  All arithmetic is FP32; each output is rounded once (E4M3:
// times the reciprocal of the cache's scale, nearest even, saturated at 448).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moedec {

namespace {

constexpr int ROPE_THREADS = 256;  // at most

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
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)from_f<BF>(f[2 * i]) | (uint32_t)from_f<BF>(f[2 * i + 1]) << 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&f)[8], float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = (uint32_t)e4m3_pair(f[4 * i] * inv, f[4 * i + 1] * inv) |
               (uint32_t)e4m3_pair(f[4 * i + 2] * inv, f[4 * i + 3] * inv) << 16;
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <bool BF>
__device__ __forceinline__ void floats8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = to_f<BF>((uint16_t)w[i]);
        f[2 * i + 1] = to_f<BF>((uint16_t)(w[i] >> 16));
    }
}

// What a token needs before its heads: the sines of its pairs (by pair) and
// its cache row, by the block's threads into shared memory.
struct RopeToken {
    float2 cs[MOE_ROPE_MAX_DIM / 2];
    int64_t page, row;  // page -1: not written
};
__device__ __forceinline__ void rope_token(const RopeArgs& a, int tok, const uint64_t* F, RopeToken& s) {
    const int half = a.rot / 2;
    const uint64_t pos = (uint64_t)(int64_t)a.positions[tok];
    for (int i = threadIdx.x; i < half; i += blockDim.x) {
        const float x = (float)(int32_t)((pos * F[i]) >> 32) * 4.656612873077393e-10f;  // 2^-31: half turns
        float sn, c;
        sincospif(x, &sn, &c);
        s.cs[i] = make_float2(c * a.mscale, sn * a.mscale);
    }
    if (threadIdx.x == blockDim.x - 1) {
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
        s.page = page;
        s.row = row;
    }
}
// The pairs' turns per position as 64-bit fractions.
__device__ __forceinline__ void rope_turns(const RopeArgs& a, uint64_t* F) {
    for (int i = threadIdx.x; i < a.rot / 2; i += blockDim.x) {
        double turns = a.freqs[i] * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= floor(turns);
        F[i] = (uint64_t)(turns * 18446744073709551616.0);
    }
}

// Head h of a token, counted over queries, keys, values: where it lies and
// where it goes (dst null: nowhere).
struct RopeHead {
    const uint16_t* src;
    uint8_t* dst;
    float inv;   // reciprocal scale of an E4M3 cache
    bool cache, turn;
};
template <int CES>
__device__ __forceinline__ RopeHead rope_head(const RopeArgs& a, int tok, int h, int64_t page, int64_t row) {
    if (h < a.Hq)
        return {static_cast<const uint16_t*>(a.q) + tok * a.q_st + h * a.q_sh,
                static_cast<uint8_t*>(a.q_out) + (tok * a.qo_st + h * a.qo_sh) * 2, 1.f, false, true};
    h -= a.Hq;
    if (h < a.Hkv)
        return {static_cast<const uint16_t*>(a.k) + tok * a.k_st + h * a.k_sh,
                page < 0 ? nullptr : static_cast<uint8_t*>(a.kc) + (page * a.kc_sp + row * a.kc_st + h * a.kc_sh) * CES,
                a.k_inv, true, true};
    h -= a.Hkv;
    return {static_cast<const uint16_t*>(a.v) + tok * a.v_st + h * a.v_sh,
            page < 0 ? nullptr : static_cast<uint8_t*>(a.vc) + (page * a.vc_sp + row * a.vc_st + h * a.vc_sh) * CES,
            a.v_inv, true, false};
}

}  // namespace

// Rows 16-byte aligned, D and the rotated halves (or pairs) in whole vectors
// of 8.  units: places of a head -- rot/16 of eight pairs (i, i + rot/2), or
// rot/8 of four adjacent pairs (INTER), then the vectors beyond rot.
template <bool BF, bool E4, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, 3) rope_append_kernel(const __grid_constant__ RopeArgs a, int units) {
    __shared__ RopeToken sm_tok[2];
    __shared__ uint64_t sm_turns[MOE_ROPE_MAX_DIM / 2];
    constexpr int CES = E4 ? 1 : 2;
    constexpr int PAIRS = INTER ? 4 : 8;
    constexpr int AHEAD = INTER ? 4 : 2;  // heads whose loads (64 bytes of them) are issued together
    const int half = a.rot / 2;
    const int rot_units = INTER ? a.rot / 8 : a.rot / 16;
    const int group = threadIdx.x / units, unit = threadIdx.x - group * units;
    const int groups = blockDim.x / units;
    const bool turns = unit < rot_units, two = turns && !INTER;
    const int dim = turns ? unit * 8 : a.rot + (unit - rot_units) * 8;
    const int heads = group < groups ? a.Hq + 2 * a.Hkv : 0;
    rope_turns(a, sm_turns);
    __syncthreads();
    int buf = 0;
    for (int tok = blockIdx.x; tok < a.T; tok += gridDim.x, buf ^= 1) {
        uint4 x[AHEAD], y[AHEAD];
        auto load = [&](int h0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int h = h0 + i * groups;
                if (h < heads) {
                    const uint16_t* src = rope_head<CES>(a, tok, h, -1, 0).src + dim;
                    x[i] = *reinterpret_cast<const uint4*>(src);
                    if (two) y[i] = *reinterpret_cast<const uint4*>(src + half);
                }
            }
        };
        load(group);
        rope_token(a, tok, sm_turns, sm_tok[buf]);
        __syncthreads();  // (the other buffer's readers are past: one token apart)
        const int64_t page = sm_tok[buf].page, row = sm_tok[buf].row;
        float2 cs[PAIRS];
        if (turns)
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) cs[p] = sm_tok[buf].cs[unit * PAIRS + p];
        for (int h0 = group; h0 < heads; h0 += AHEAD * groups) {
            if (h0 != group) load(h0);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int h = h0 + i * groups;
                if (h >= heads) continue;
                const RopeHead hd = rope_head<CES>(a, tok, h, page, row);
                if (!hd.dst) continue;
                float f[8], e[8];
                floats8<BF>(x[i], f);
                if (two) floats8<BF>(y[i], e);
                if (turns && hd.turn) {
                    if (INTER) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const float u = f[2 * p], v = f[2 * p + 1];
                            f[2 * p] = u * cs[p].x - v * cs[p].y;
                            f[2 * p + 1] = v * cs[p].x + u * cs[p].y;
                        }
                    } else {
#pragma unroll
                        for (int p = 0; p < 8; ++p) {
                            const float u = f[p], v = e[p];
                            f[p] = u * cs[p % PAIRS].x - v * cs[p % PAIRS].y;
                            e[p] = v * cs[p % PAIRS].x + u * cs[p % PAIRS].y;
                        }
                    }
                }
                if (E4 && hd.cache) {
                    store8_e4m3(hd.dst + dim, f, hd.inv);
                    if (two) store8_e4m3(hd.dst + dim + half, e, hd.inv);
                } else {
                    store8<BF>(reinterpret_cast<uint16_t*>(hd.dst) + dim, f);
                    if (two) store8<BF>(reinterpret_cast<uint16_t*>(hd.dst) + dim + half, e);
                }
            }
        }
    }
}

// Any alignment: one pair or element per thread.
template <bool BF, bool E4>
__global__ void __launch_bounds__(ROPE_THREADS) rope_append_any_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ RopeToken sm_tok[2];
    __shared__ uint64_t sm_turns[MOE_ROPE_MAX_DIM / 2];
    const int half = a.rot / 2;
    const int units = half + a.D - a.rot;
    const int total = (a.Hq + 2 * a.Hkv) * units;
    rope_turns(a, sm_turns);
    __syncthreads();
    int buf = 0;
    for (int tok = blockIdx.x; tok < a.T; tok += gridDim.x, buf ^= 1) {
        rope_token(a, tok, sm_turns, sm_tok[buf]);
        __syncthreads();
        for (int i = threadIdx.x; i < total; i += blockDim.x) {
            const int h = i / units, unit = i - h * units;
            const RopeHead hd = rope_head<E4 ? 1 : 2>(a, tok, h, sm_tok[buf].page, sm_tok[buf].row);
            if (!hd.dst) continue;
            auto put = [&](int d, float f) {
                if (E4 && hd.cache)
                    hd.dst[d] = (uint8_t)e4m3_pair(f * hd.inv, 0.f);
                else
                    reinterpret_cast<uint16_t*>(hd.dst)[d] = from_f<BF>(f);
            };
            if (unit < half) {
                const int d0 = a.interleaved ? 2 * unit : unit, d1 = a.interleaved ? d0 + 1 : unit + half;
                const float u = to_f<BF>(hd.src[d0]), v = to_f<BF>(hd.src[d1]);
                const float2 cs = hd.turn ? sm_tok[buf].cs[unit] : make_float2(1.f, 0.f);
                put(d0, hd.turn ? u * cs.x - v * cs.y : u);
                put(d1, hd.turn ? v * cs.x + u * cs.y : v);
            } else {
                const int d = a.rot + unit - half;
                put(d, to_f<BF>(hd.src[d]));
            }
        }
    }
}

template <bool BF, bool E4>
static cudaError_t launch_rope(const RopeArgs& a, const DeviceInfo& di, cudaStream_t st) {
    auto al = [](const void* p, int64_t s0, int64_t s1, int64_t s2) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 % 8 == 0 && s1 % 8 == 0 && s2 % 8 == 0;
    };
    const bool vec = a.D % 8 == 0 && a.rot % (a.interleaved ? 8 : 16) == 0 && al(a.q, a.q_st, a.q_sh, 0) &&
                     al(a.k, a.k_st, a.k_sh, 0) && al(a.v, a.v_st, a.v_sh, 0) && al(a.q_out, a.qo_st, a.qo_sh, 0) &&
                     al(a.kc, a.kc_sp, a.kc_st, a.kc_sh) && al(a.vc, a.vc_sp, a.vc_st, a.vc_sh);
    if (vec) {
        // threads for all the heads at once, between 64 and 256
        const int units = (a.interleaved ? a.rot / 8 : a.rot / 16) + (a.D - a.rot) / 8;
        const int64_t want = (int64_t)units * (a.Hq + 2 * a.Hkv);
        const int threads = want <= 64 ? 64 : want <= 128 ? 128 : ROPE_THREADS;
        const int grid = std::min(a.T, di.sm_count * (3 * ROPE_THREADS / threads));
        if (a.interleaved)
            rope_append_kernel<BF, E4, true><<<grid, threads, 0, st>>>(a, units);
        else
            rope_append_kernel<BF, E4, false><<<grid, threads, 0, st>>>(a, units);
    } else {
        rope_append_any_kernel<BF, E4><<<std::min(a.T, di.sm_count * 8), ROPE_THREADS, 0, st>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_rope_append(RopeArgs a, int dtype, int cache_dtype, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    a.err = di.err_word;
    a.k_inv = cache_dtype == MOE_E4M3 ? 1.f / a.k_scale : 1.f;
    a.v_inv = cache_dtype == MOE_E4M3 ? 1.f / a.v_scale : 1.f;
    if (cache_dtype == MOE_E4M3) return dtype == MOE_BF16 ? launch_rope<true, true>(a, di, st) : launch_rope<false, true>(a, di, st);
    return dtype == MOE_BF16 ? launch_rope<true, false>(a, di, st) : launch_rope<false, false>(a, di, st);
}

}  // namespace moedec
