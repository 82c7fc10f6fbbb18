// rope.cu -- rotary positions on the query and key heads of new tokens,
// fused with writing the rotated keys and the values into a paged cache.
//
// Mathematics.  Pair i of a head's first `rot` dims is (x_i, x_{i+rot/2}) in
// the half layout and (x_{2i}, x_{2i+1}) interleaved; with a = pos * f_i,
//   (x, y) -> mscale * (x cos a - y sin a,  y cos a + x sin a).
// The angle is reduced exactly: f_i / 2 pi is taken modulo 1 as a 64-bit
// fraction F_i of a turn (FP64, once per block), and pos * F_i wraps modulo
// 2^64, that is modulo a whole turn: the phase is right to 2^-32 turns at a
// position of 2^20, to 2^-23 at one of 2^31 (FP64's rounding of F_i), where an
// FP32 product would be off by radians.  Its top 32 bits, as a signed fraction
// of half a turn, become a float (2^-26 turns off at most) for sincospif.
//
// Bound: HBM, each element in and out once (16384 tokens of 64 + 8 + 8 heads
// of 128: 671 MB, 107 us, 6.3 TB/s).  One block takes one or a few tokens at a
// time (blocks stride over the tokens): their rot/2 sines go to shared memory
// once and serve every head.  A thread keeps one place within a head (a
// 16-byte vector, or the two vectors of eight rotated pairs) of the same heads
// throughout, so that addresses only move on, and the heads' loads are on
// their way before the sines are made.  All arithmetic is FP32; each output is
// rounded once (E4M3: times the reciprocal of the cache's scale, nearest even,
// saturated at 448).
#include <algorithm>

#include "block_common.cuh"
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
__device__ __forceinline__ float2 rope_sine(int position, uint64_t turns, float mscale) {
    const uint64_t phase = (uint64_t)(int64_t)position * turns;
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    return make_float2(c * mscale, s * mscale);
}
struct RopeToken {
    float2 cs[MOE_ROPE_MAX_DIM / 2];
    int64_t page, row;  // page -1: not written
};
__device__ __forceinline__ void rope_token(const RopeArgs& a, int position, int64_t slot, const uint64_t* F, RopeToken& s) {
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < half; i += blockDim.x) s.cs[i] = rope_sine(position, F[i], a.mscale);
    if (threadIdx.x == blockDim.x - 1) {
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

// The two vector kernels want rows 16-byte aligned, D and the rotated halves
// (or pairs) in whole vectors of 8.  units: places of a head -- rot/16 of
// eight pairs (i, i + rot/2), or rot/8 of four adjacent pairs (INTER), then
// the vectors beyond rot.

// One place of a head: eight elements, and their pairs' other halves (half
// layout: Place::two), rotated by the sines of its pairs.
template <bool BF, bool INTER>
struct Place {
    static constexpr int PAIRS = INTER ? 4 : 8;
    uint4 x, y;
    __device__ __forceinline__ void load(const uint16_t* p, bool two, int half) {
        x = *reinterpret_cast<const uint4*>(p);
        if (two) y = *reinterpret_cast<const uint4*>(p + half);
    }
    __device__ __forceinline__ void floats(float (&f)[8], float (&e)[8], bool two) const {
        floats8<BF>(x, f);
        if (two) floats8<BF>(y, e);
    }
    static __device__ __forceinline__ void rotate(float (&f)[8], float (&e)[8], const float2* cs) {
        if (INTER) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float s = f[2 * p], t = f[2 * p + 1];
                f[2 * p] = s * cs[p].x - t * cs[p].y;
                f[2 * p + 1] = t * cs[p].x + s * cs[p].y;
            }
        } else {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const float s = f[p], t = e[p];
                f[p] = s * cs[p % PAIRS].x - t * cs[p % PAIRS].y;
                e[p] = t * cs[p % PAIRS].x + s * cs[p % PAIRS].y;
            }
        }
    }
};
template <bool BF>
__device__ __forceinline__ void put_half(uint16_t* p, const float (&f)[8], const float (&e)[8], bool two, int half) {
    store8<BF>(p, f);
    if (two) store8<BF>(p + half, e);
}
template <bool BF, bool E4>
__device__ __forceinline__ void put_cache(uint8_t* p, const float (&f)[8], const float (&e)[8], bool two, int half, float inv) {
    if (E4) {
        store8_e4m3(p, f, inv);
        if (two) store8_e4m3(p + half, e, inv);
    } else {
        put_half<BF>(reinterpret_cast<uint16_t*>(p), f, e, two, half);
    }
}

// Many heads: one token at a time, each thread in one place of every
// (256 / units)-th head, its sines in registers.
template <bool BF, bool E4, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, INTER ? 3 : 2)
    rope_heads_kernel(const __grid_constant__ RopeArgs a, int units) {
    __shared__ RopeToken sm_tok[2];
    __shared__ uint64_t sm_turns[MOE_ROPE_MAX_DIM / 2];
    after_previous();
    using P = Place<BF, INTER>;
    constexpr int CES = E4 ? 1 : 2;
    constexpr int AHEAD = INTER ? 4 : 2;  // query heads whose loads are issued together
    const int half = a.rot / 2;
    const int rot_units = INTER ? a.rot / 8 : a.rot / 16;
    const int group = threadIdx.x / units, unit = threadIdx.x - group * units;
    const int groups = ROPE_THREADS / units;
    const bool turns = unit < rot_units, two = turns && !INTER;
    const int dim = turns ? unit * 8 : a.rot + (unit - rot_units) * 8;
    const int nq = group < groups ? a.Hq : 0, nkv = group < groups ? a.Hkv : 0;
    // this thread's place in its first head, and steps to its next one
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + blockIdx.x * a.q_st + group * a.q_sh + dim;
    const uint16_t* k = static_cast<const uint16_t*>(a.k) + blockIdx.x * a.k_st + group * a.k_sh + dim;
    const uint16_t* v = static_cast<const uint16_t*>(a.v) + blockIdx.x * a.v_st + group * a.v_sh + dim;
    uint16_t* qo = static_cast<uint16_t*>(a.q_out) + blockIdx.x * a.qo_st + group * a.qo_sh + dim;
    const int64_t q_step = groups * a.q_sh, qo_step = groups * a.qo_sh;
    float2 cs[P::PAIRS];

    // a token's position and slot are loaded while the one before is worked on
    int position = a.positions[blockIdx.x];
    int64_t slot = a.slots[blockIdx.x];
    rope_turns(a, sm_turns);
    __syncthreads();
    int buf = 0;
    const uint32_t T = a.T;  // (unsigned: a token number past T may pass 2^31)
    for (uint32_t tok = blockIdx.x; tok < T; tok += gridDim.x, buf ^= 1) {
        // the first heads are on their way while the sines are made
        P pq[AHEAD], pk, pv;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (group + i * groups < nq) pq[i].load(q + i * q_step, two, half);
        if (group < nkv) {
            pk.load(k, two, half);
            pv.load(v, two, half);
        }
        rope_token(a, position, slot, sm_turns, sm_tok[buf]);
        if (tok + gridDim.x < T) {
            position = a.positions[tok + gridDim.x];
            slot = a.slots[tok + gridDim.x];
        }
        __syncthreads();  // (the other buffer's readers are past: one token apart)
        const int64_t page = sm_tok[buf].page, row = sm_tok[buf].row;
        if (turns)
#pragma unroll
            for (int p = 0; p < P::PAIRS; ++p) cs[p] = sm_tok[buf].cs[unit * P::PAIRS + p];
        const uint16_t* qh = q;
        uint16_t* qoh = qo;
        float f[8], e[8];
        for (int h = group; h < nq; h += AHEAD * groups) {
            if (h != group)
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (h + i * groups < nq) pq[i].load(qh + i * q_step, two, half);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (h + i * groups < nq) {
                    pq[i].floats(f, e, two);
                    if (turns) P::rotate(f, e, cs);
                    put_half<BF>(qoh + i * qo_step, f, e, two, half);
                }
            qh += AHEAD * q_step;
            qoh += AHEAD * qo_step;
        }
        if (page >= 0) {
            for (int h = group; h < nkv; h += groups) {
                if (h != group) {
                    pk.load(k + (h - group) * a.k_sh, two, half);
                    pv.load(v + (h - group) * a.v_sh, two, half);
                }
                pk.floats(f, e, two);
                if (turns) P::rotate(f, e, cs);
                put_cache<BF, E4>(static_cast<uint8_t*>(a.kc) + (page * a.kc_sp + row * a.kc_st + h * a.kc_sh + dim) * CES, f, e,
                                  two, half, a.k_inv);
                pv.floats(f, e, two);
                put_cache<BF, E4>(static_cast<uint8_t*>(a.vc) + (page * a.vc_sp + row * a.vc_st + h * a.vc_sh + dim) * CES, f, e,
                                  two, half, a.v_inv);
            }
        }
        q += gridDim.x * a.q_st;
        k += gridDim.x * a.k_st;
        v += gridDim.x * a.v_st;
        qo += gridDim.x * a.qo_st;
    }
}

// Fewer heads: `toks` tokens at a time, whose heads (queries, keys, values)
// are dealt to groups of `units` threads, JOBS to each at most.  A thread's
// jobs stay the same heads of the block's first, second .. token throughout.
// (Half layout: four jobs of 32 bytes in two blocks per SM, 66 us at 16384
// tokens of 32 / 4 heads of 128, 336 MB, 5.1 TB/s; two in three blocks 81, three
// in two 75.)
constexpr int ROPE_SINES = 512;  // pairs of a block's tokens at most
constexpr int ROPE_TOKS = 16;
constexpr int ROPE_JOBS = 4;
template <bool BF, bool E4, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, INTER ? 3 : 2)
    rope_tokens_kernel(const __grid_constant__ RopeArgs a, int units, int toks) {
    after_previous();
    using P = Place<BF, INTER>;
    constexpr int JOBS = ROPE_JOBS;
    constexpr int CES = E4 ? 1 : 2;
    __shared__ __align__(16) float2 sm_cs[2][ROPE_SINES];
    __shared__ uint64_t sm_turns[MOE_ROPE_MAX_DIM / 2];
    // Offsets of the token's row in the K and V caches; -1: none.  Three places:
    // a round's are read after its barrier, the next round's are written before
    // it, and the round after that is written while slower warps still read.
    __shared__ int64_t sm_row[3][ROPE_TOKS][2];
    __shared__ int sm_pos[2][ROPE_TOKS];
    const int tid = threadIdx.x;
    const int half = a.rot / 2;
    const int rot_units = INTER ? a.rot / 8 : a.rot / 16;
    const int group = tid / units, unit = tid - group * units;
    const int groups = ROPE_THREADS / units;
    const bool turns = unit < rot_units, two = turns && !INTER;
    const int dim = turns ? unit * 8 : a.rot + (unit - rot_units) * 8;
    const int heads = a.Hq + 2 * a.Hkv;

    const int64_t stride = (int64_t)gridDim.x * toks;
    // a token's position and slot: loaded two rounds ahead, put into shared memory one ahead
    auto put_token = [&](int b, int at, int64_t tok, int position, int64_t slot) {
        int64_t kr = -1, vr = -1;
        if (tok < a.T && slot >= 0) {
            const int64_t page = slot / a.page, row = slot - page * a.page;
            if (page < a.num_pages) {
                kr = page * a.kc_sp + row * a.kc_st;
                vr = page * a.vc_sp + row * a.vc_st;
            } else {
                atomicOr(a.err, MOE_DEVERR_PAGE);
            }
        }
        sm_row[at][tid][0] = kr;
        sm_row[at][tid][1] = vr;
        sm_pos[b][tid] = position;
    };
    int position = 0;
    int64_t slot = -1;
    auto load_token = [&](int64_t tok) {
        if (tok < a.T) {
            position = a.positions[tok];
            slot = a.slots[tok];
        }
    };
    const int64_t first = (int64_t)blockIdx.x * toks;
    if (tid < toks) {
        load_token(first + tid);
        put_token(0, 0, first + tid, position, slot);
        load_token(first + stride + tid);
    }
    const uint16_t* src[JOBS];
    uint8_t* dst[JOBS];         // the query's place (moving on); the head's place in a cache row
    int64_t src_step[JOBS];
    int kind[JOBS], tokl[JOBS];  // 0 query, 1 key, 2 value, 3 nothing
#pragma unroll
    for (int j = 0; j < JOBS; ++j) {
        const int hh = group + j * groups;
        const int tl = hh / heads, h = hh - tl * heads;
        tokl[j] = tl;
        kind[j] = group >= groups || tl >= toks ? 3 : h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;
        const int64_t tok = first + tl;
        if (kind[j] == 0) {
            src[j] = static_cast<const uint16_t*>(a.q) + tok * a.q_st + h * a.q_sh + dim;
            dst[j] = static_cast<uint8_t*>(a.q_out) + (tok * a.qo_st + h * a.qo_sh + dim) * 2;
            src_step[j] = stride * a.q_st;
        } else if (kind[j] == 1) {
            src[j] = static_cast<const uint16_t*>(a.k) + tok * a.k_st + (h - a.Hq) * a.k_sh + dim;
            dst[j] = static_cast<uint8_t*>(a.kc) + ((h - a.Hq) * a.kc_sh + dim) * CES;
            src_step[j] = stride * a.k_st;
        } else {
            src[j] = static_cast<const uint16_t*>(a.v) + tok * a.v_st + (h - a.Hq - a.Hkv) * a.v_sh + dim;
            dst[j] = static_cast<uint8_t*>(a.vc) + ((h - a.Hq - a.Hkv) * a.vc_sh + dim) * CES;
            src_step[j] = stride * a.v_st;
        }
    }
    const int64_t qo_step = stride * a.qo_st * 2;
    rope_turns(a, sm_turns);
    __syncthreads();

    int buf = 0, at = 0;  // places of this round's sines and positions, and of its rows
    for (int64_t t0 = first; t0 < a.T; t0 += stride, buf ^= 1) {
        const int at_next = at == 2 ? 0 : at + 1;
        P place[JOBS];
#pragma unroll
        for (int j = 0; j < JOBS; ++j)
            if (kind[j] != 3 && t0 + tokl[j] < a.T) place[j].load(src[j], two, half);
        // (half layout: two pairs of one unit, then of the next, so that a warp's
        // reads of 16 bytes by consecutive units are consecutive; it took 8 of 90
        // us off 16384 tokens of 32 / 4 heads of 128.  The four pairs of an interleaved
        // unit meet two-way conflicts as they lie, which costs less than the
        // registers of the other order: 59 against 65 us at 85836 of 4 / 1.)
        for (int i = tid; i < toks * half; i += ROPE_THREADS) {
            const int tl = i / half, pair = i - tl * half, r = pair % P::PAIRS;
            sm_cs[buf][tl * half + (INTER ? pair : (r >> 1) * 2 * rot_units + pair / P::PAIRS * 2 + (r & 1))] =
                rope_sine(sm_pos[buf][tl], sm_turns[pair], a.mscale);
        }
        if (tid < toks) {
            put_token(buf ^ 1, at_next, t0 + stride + tid, position, slot);
            load_token(t0 + 2 * stride + tid);
        }
        // One barrier a round.  Sines: written before it and read after it, so
        // the readers of this place, two rounds back, are past the barrier
        // between.  Positions: read before it, written for the next round
        // before it, in the place that was read before the last one.  Rows:
        // written for the next round before it, in the place that was read
        // two rounds back, before the last barrier.
        __syncthreads();
#pragma unroll
        for (int j = 0; j < JOBS; ++j) {
            if (kind[j] != 3 && t0 + tokl[j] < a.T) {
                float f[8], e[8];
                place[j].floats(f, e, two);
                if (INTER && turns && kind[j] != 2) P::rotate(f, e, sm_cs[buf] + tokl[j] * half + unit * P::PAIRS);
                if (!INTER && turns && kind[j] != 2) {
                    float2 cs[P::PAIRS];
#pragma unroll
                    for (int p = 0; p < P::PAIRS / 2; ++p) {
                        const float4 c =
                            *reinterpret_cast<const float4*>(&sm_cs[buf][tokl[j] * half + (p * rot_units + unit) * 2]);
                        cs[2 * p] = make_float2(c.x, c.y);
                        cs[2 * p + 1] = make_float2(c.z, c.w);
                    }
                    P::rotate(f, e, cs);
                }
                if (kind[j] == 0) {
                    put_half<BF>(reinterpret_cast<uint16_t*>(dst[j]), f, e, two, half);
                    dst[j] += qo_step;
                } else {
                    const int64_t row = sm_row[at][tokl[j]][kind[j] - 1];
                    if (row >= 0) put_cache<BF, E4>(dst[j] + row * CES, f, e, two, half, kind[j] == 1 ? a.k_inv : a.v_inv);
                }
            }
            src[j] += src_step[j];
        }
        at = at_next;
    }
}

// Any alignment: one pair or element per thread.
template <bool BF, bool E4>
__global__ void __launch_bounds__(ROPE_THREADS) rope_append_any_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ RopeToken sm_tok[2];
    __shared__ uint64_t sm_turns[MOE_ROPE_MAX_DIM / 2];
    after_previous();
    const int half = a.rot / 2;
    const int units = half + a.D - a.rot;
    const int total = (a.Hq + 2 * a.Hkv) * units;
    rope_turns(a, sm_turns);
    __syncthreads();
    int buf = 0;
    const uint32_t T = a.T;  // (unsigned: a token number past T may pass 2^31)
    for (uint32_t tok = blockIdx.x; tok < T; tok += gridDim.x, buf ^= 1) {
        rope_token(a, a.positions[tok], a.slots[tok], sm_turns, sm_tok[buf]);
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
        const int units = (a.interleaved ? a.rot / 8 : a.rot / 16) + (a.D - a.rot) / 8;
        const int jobs = ROPE_THREADS / units * ROPE_JOBS, heads = a.Hq + 2 * a.Hkv;
        if (heads > jobs) {
            const int grid = std::min(a.T, di.sm_count * (a.interleaved ? 3 : 2));
            if (a.interleaved)
                return launch_after(rope_heads_kernel<BF, E4, true>, dim3(grid), ROPE_THREADS, 0, st, a, units);
            return launch_after(rope_heads_kernel<BF, E4, false>, dim3(grid), ROPE_THREADS, 0, st, a, units);
        }
        // as many tokens as the threads have jobs for, once every block has some
        const int blocks = di.sm_count * (a.interleaved ? 3 : 2);
        int toks = std::min(jobs / heads, std::min(ROPE_TOKS, a.T / blocks));
        if (a.rot) toks = std::min(toks, 2 * ROPE_SINES / a.rot);
        toks = std::max(toks, 1);
        const int grid = std::min((a.T - 1) / toks + 1, blocks);
        if (a.interleaved)
            return launch_after(rope_tokens_kernel<BF, E4, true>, dim3(grid), ROPE_THREADS, 0, st, a, units, toks);
        return launch_after(rope_tokens_kernel<BF, E4, false>, dim3(grid), ROPE_THREADS, 0, st, a, units, toks);
    }
    return launch_after(rope_append_any_kernel<BF, E4>, dim3(std::min(a.T, di.sm_count * 8)), ROPE_THREADS, 0, st, a);
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
