// router_grouped.cu -- routing with a bias for balance and with groups of
// experts: per token, scores s (softmax or sigmoid of its E logits), keys
// s + bias that decide, the best groups of experts by their best key or the
// sum of their two best, the k largest keys within those groups (ties: the
// lower expert first), and weights from the scores alone.
//
// Which of two keys is larger is decided for the real numbers, not for their
// FP32 roundings: FP32 keys choose, and where two that matter lie within their
// errors of each other, the keys of the candidates are computed again in 64 bits.
// Without a bias (or with the same one for all) the logits themselves are the
// keys, which needs no second look.
//
// One warp per token at a time, a lane holds NV consecutive logits.  Each lane
// sorts its keys (a network of maxima and minima) and leaves the list in shared
// memory; a pick is the largest of the 32 list heads, one redux instruction on
// order-preserving integers, and the next head of the list that had it.  Whose
// index a picked key had is found once, for all picks at the same time.
// Bound: latency for few tokens (33 rows of 256 experts: 4.1 us).  For many
// (65536 rows of 256, 8 groups, 8 picks, FP32: 55 us, 1.3 TB/s, BF16 52 us; the
// logits' bytes alone would take 10) the dependent steps and exchanges of the 16
// warps that an SM has room for: 2.2 of 4 instructions issue a cycle.  Shapes that
// the eight-lane kernel does not take need a warp a row: 65536 rows of 512, 10
// picks, 142 us; of 160 in 16 groups 96.
#include <algorithm>

#include "block_common.cuh"
#include "internal.h"

namespace moedec {

namespace {

constexpr int rg_warps(int nv) { return nv == 32 ? 4 : 8; }  // (48 KB hold the lists of four warps of 1024)

// Order-preserving map of floats (not NaN; the two zeros alike) to unsigned; 0 is below -inf's.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(f + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(FULL_MASK, v); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    return v;
}

template <int DT>
__device__ __forceinline__ float logit_at(const void* row, int e) {
    if (DT == MOE_F32) return static_cast<const float*>(row)[e];
    const uint16_t h = static_cast<const uint16_t*>(row)[e];
    if (DT == MOE_BF16) return __uint_as_float((uint32_t)h << 16);
    return __half2float(__ushort_as_half(h));
}

__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Descending order by odd-even merges.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) { return min(a, b); }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
template <int N, class T>
__device__ __forceinline__ void sort_down(T (&v)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const T a = v[i + j], b = v[i + j + k];
                        v[i + j] = larger(a, b);
                        v[i + j + k] = smaller(a, b);
                    }
}

// NV consecutive logits from expert e0 on, -inf beyond E and for NaN.
template <int NV, int DT>
__device__ __forceinline__ void load_logits(const void* row, int e0, int E, bool vec, float (&x)[NV]) {
    if (vec) {  // E a multiple of 4, rows aligned to four logits
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
            uint32_t w[4] = {0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u};
            if (e0 + i < E) {
                if (DT == MOE_F32) {
                    const uint4 v = ld_128(static_cast<const float*>(row) + e0 + i);
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + e0 + i);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t h = (k < 2 ? v.x : v.y) >> (k & 1) * 16 & 0xffffu;
                        w[k] = DT == MOE_BF16 ? h << 16 : __float_as_uint(__half2float(__ushort_as_half((uint16_t)h)));
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i + k] = __uint_as_float(w[k]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = e0 + i < E ? logit_at<DT>(row, e0 + i) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = fmaxf(x[i], -INFINITY);  // (of NaN: -inf)
}

// What FP32 scores are off by at most, in units of 2^-24.  Sigmoid, of a value
// s <= 1: 2 for the quotient, 1 for the sum 1 + e, and s (1 - s) times the
// relative error of e, 4 of exp2 and 1.5 |x| of its argument: 1 + 0.4; under
// 5.5.  Softmax, relative to a score of at most 1 / total: 4 of exp2, and 2.23
// |x - m| of its argument (a difference, a product and the constant's own 0.23;
// a score times |x - m| is at most 0.37 / total); of the sum 4 of exp2, 2.23
// times the mean of |x - m| by the scores (at most 4.44 for 1024 experts), 37 of
// its additions; 2 of the quotient; under 58.
__device__ __forceinline__ float score_error(bool softmax, float total) { return softmax ? 0x40p-24f / total : 0x5.8p-24f; }

// What a group's worth is off by at most: its keys' scores, and a rounding of
// each key and of their sum.  The keys may cancel (biases of either sign), so
// their sizes count and not their sum's.
__device__ __forceinline__ float worth_error(float worth, float best, float second, float tau_s) {
    return fabsf(worth) < INFINITY ? 2.f * tau_s + 0x1p-22f * (fabsf(best) + fabsf(second)) : 0.f;
}

// A score in 64 bits; `m` and `total` are the row's (softmax).
__device__ __forceinline__ double score64(const RouterGroupedArgs& a, float x, double m, double total) {
    return a.score == MOE_ROUTER_SOFTMAX ? exp((double)x - m) / total : 1.0 / (1.0 + exp(-(double)x));
}

}  // namespace

// What is the same for all rows of a call.
template <int NV>
struct RowPlan {
    float bias[NV];  // of the lane's experts
    bool same_bias;  // one bias for all experts changes no order
    __device__ __forceinline__ explicit RowPlan(const RouterGroupedArgs& a) {
        const int e0 = (threadIdx.x & 31) * NV;
        const float b0 = a.bias ? a.bias[0] : 0.f;
        same_bias = true;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            bias[i] = a.bias && e0 + i < a.E ? a.bias[e0 + i] : 0.f;
            if (e0 + i < a.E && bias[i] != b0) same_bias = false;
        }
        same_bias = __all_sync(FULL_MASK, same_bias) && fabsf(b0) < INFINITY;
    }
};

// Row t by a whole warp.  sk [32 NV]: keys by expert; lists [32][NV + 1]: each
// lane's in descending order, and a 0 at the end.
template <int NV, int DT>
__device__ __forceinline__ void route_row(const RouterGroupedArgs& a, int64_t t, const RowPlan<NV>& plan, uint32_t* sk,
                                          uint32_t* lists) {
    const int lane = threadIdx.x & 31;
    const int E = a.E, k = a.k, e0 = lane * NV;
    uint32_t* const list = lists + lane * (NV + 1);
    const float(&bias)[NV] = plan.bias;
    const bool same_bias = plan.same_bias;
    const bool softmax = a.score == MOE_ROUTER_SOFTMAX;
    const bool narrow = a.top_groups < a.groups;
    const int gsize = E / a.groups;
    // lanes of a group, where each group is a power of two of whole lanes
    const int q = gsize % NV ? 0 : gsize / NV;
    const bool whole_lanes = q > 0 && (q & (q - 1)) == 0;
    const bool top2 = a.group_score == MOE_ROUTER_GROUP_TOP2;
    const bool by_logit = same_bias && !top2;

    const void* row = static_cast<const uint8_t*>(a.logits) + t * a.stride * (DT == MOE_F32 ? 4 : 2);
    float x[NV];
    load_logits<NV, DT>(row, e0, E, a.vec, x);
    // scores
    float m = 0.f, total = 1.f, s[NV];
    if (softmax) {
        float u = x[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) u = fmaxf(u, x[i]);
        m = unordered(warp_max(ordered(u)));
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            s[i] = x[i] == -INFINITY ? 0.f : exp2_ftz((x[i] - m) * 1.44269504f);
            sum += s[i];
        }
        total = warp_sum(sum);
        const float inv = 1.f / total;
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] *= inv;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = rcp_fast(1.f + exp2_ftz(x[i] * -1.44269504f));
    }
    const float tau_s = score_error(softmax, total);
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float f = same_bias ? x[i] : s[i] + bias[i];
        key[i] = x[i] > -INFINITY && f > -INFINITY ? ordered(f) : 0u;
    }

    double m64 = 0., total64 = 1.;
    bool have64 = false;
    auto row64 = [&]() {  // the softmax's sum in 64 bits
        if (have64 || !softmax) return;
        m64 = m;
        double d = 0.;
#pragma unroll 1
        for (int i = 0; i < NV; ++i)
            if (e0 + i < E) {
                const float v = logit_at<DT>(row, e0 + i);
                if (v > -INFINITY) d += exp((double)v - m64);
            }
        total64 = warp_sum(d);
        have64 = true;
    };

    if (narrow) {
        // a group's worth: lane g has group g's
        float best = -INFINITY, second = -INFINITY;
        auto see = [&](float v) {
            second = fmaxf(second, fminf(best, v));
            best = fmaxf(best, v);
        };
        auto part = [&](int i) {  // what counts of the lane's element i
            return key[i] == 0u ? -INFINITY : by_logit ? x[i] : same_bias ? s[i] : s[i] + bias[i];
        };
        if (whole_lanes) {
#pragma unroll
            for (int i = 0; i < NV; ++i) see(part(i));
            for (int o = 1; o < q; o *= 2) {
                const float b2 = __shfl_xor_sync(FULL_MASK, best, o), s2 = __shfl_xor_sync(FULL_MASK, second, o);
                second = fmaxf(fmaxf(second, s2), fminf(best, b2));
                best = fmaxf(best, b2);
            }
            best = __shfl_sync(FULL_MASK, best, lane * q & 31);
            second = __shfl_sync(FULL_MASK, second, lane * q & 31);
        } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NV; ++i) sk[e0 + i] = __float_as_uint(part(i));
            __syncwarp();
            if (lane < a.groups) {
                int at = lane % gsize;  // (lanes begin at different places: other banks)
                for (int i = 0; i < gsize; ++i) {
                    see(__uint_as_float(sk[lane * gsize + at]));
                    if (++at == gsize) at = 0;
                }
            }
        }
        float worth = top2 ? best + second : best;
        if (!(worth >= -INFINITY)) worth = -INFINITY;
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const float o = __shfl_sync(FULL_MASK, worth, g);
            rank += o > worth || (o == worth && g < lane);
        }
        bool in = lane < a.groups && rank < a.top_groups;
        if (!by_logit) {
            // the border between the least that a group in may be worth and the
            // most that one out may (infinite: whatever its neighbours)
            const float err = worth_error(worth, best, top2 ? second : 0.f, tau_s);
            const float last = unordered(~warp_max(in ? ~ordered(worth - err) : 0u));
            const float next = unordered(warp_max(lane < a.groups && !in ? ordered(worth + err) : 0u));
            if (last <= next && next > -INFINITY && last < INFINITY) {
                // the groups about it in 64 bits, the others are clearly in or out
                row64();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < NV; ++i) sk[e0 + i] = key[i];
                __syncwarp();
                double w64 = worth - err > next ? INFINITY : -INFINITY;
                const bool near = lane < a.groups && worth - err <= next && worth + err >= last;
                for (uint32_t todo = __ballot_sync(FULL_MASK, near); todo; todo &= todo - 1u) {
                    const int g = __ffs(todo) - 1;
                    double b64 = -INFINITY, s64 = -INFINITY;
                    for (int e = g * gsize + lane; e < (g + 1) * gsize; e += 32)
                        if (sk[e] != 0u) {
                            const double v = score64(a, logit_at<DT>(row, e), m64, total64) + (same_bias ? 0. : (double)a.bias[e]);
                            s64 = fmax(s64, fmin(b64, v));
                            b64 = fmax(b64, v);
                        }
#pragma unroll
                    for (int o = 16; o; o >>= 1) {
                        const double b2 = __shfl_xor_sync(FULL_MASK, b64, o), s2 = __shfl_xor_sync(FULL_MASK, s64, o);
                        s64 = fmax(fmax(s64, s2), fmin(b64, b2));
                        b64 = fmax(b64, b2);
                    }
                    if (lane == g) w64 = top2 ? b64 + s64 : b64;
                }
                rank = 0;
                for (int g = 0; g < a.groups; ++g) {
                    const double o = __shfl_sync(FULL_MASK, w64, g);
                    rank += o > w64 || (o == w64 && g < lane);
                }
                in = lane < a.groups && rank < a.top_groups;
            }
        }
        const uint32_t kept = __ballot_sync(FULL_MASK, in);
        if (whole_lanes) {
            const bool mine_in = kept >> min(31, lane / q) & 1u;
#pragma unroll
            for (int i = 0; i < NV; ++i) key[i] = mine_in ? key[i] : 0u;
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (!(kept >> min(31, (e0 + i) / gsize) & 1u)) key[i] = 0u;
        }
    }

    // the picks: lane j keeps the j-th largest key, whose it is and its place in that lane's list
    uint32_t mine;
    {
        uint32_t v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = key[i];
        sort_down(v);
        mine = v[0];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NV; ++i) list[i] = v[i];
#pragma unroll
        for (int i = 0; i < NV; ++i) sk[i * 32 + lane] = key[i];
        __syncwarp();
    }
    uint32_t pick_key = 0;
    int from = 0, place = 0, taken = 0, n = 0;
    auto next_pick = [&]() {  // false: none is left
        const uint32_t top = warp_max(mine);
        if (top == 0u) return false;
        const int owner = __ffs(__ballot_sync(FULL_MASK, mine == top)) - 1;
        const int at = __shfl_sync(FULL_MASK, taken, owner);
        if (lane == owner) mine = list[++taken];
        if (lane == n) pick_key = top, from = owner, place = at;
        ++n;
        return true;
    };
    // the expert of this lane's pick: keys of a lane's list that are equal
    // come in the order of their experts
    auto expert = [&]() {
        int above = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) above += sk[i * 32 + from] > pick_key;
        int skip = place - above, e = -1;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (sk[i * 32 + from] == pick_key && skip-- == 0) e = from * NV + i;
        return e;
    };
    const int want = same_bias ? k : min(k + 1, 32);
    while (n < want && next_pick()) {
    }
    int pick = lane < n ? expert() : -1;
    float px = pick >= 0 ? logit_at<DT>(row, pick) : 0.f;
    if (!same_bias && n > 1) {
        // neighbours within tau of each other that are not the same values
        const float f = unordered(pick_key);
        const float pb = pick >= 0 ? a.bias[pick] : 0.f;
        const float f0 = __shfl_up_sync(FULL_MASK, f, 1), x0 = __shfl_up_sync(FULL_MASK, px, 1),
                    b0 = __shfl_up_sync(FULL_MASK, pb, 1);
        const float tau = 2.f * tau_s + 0x1p-22f * fmaxf(fabsf(f), fabsf(f0));
        const bool close = lane > 0 && lane < n && f0 - f < INFINITY && f0 - f <= tau;
        bool look = __any_sync(FULL_MASK, close && !(px == x0 && pb == b0));
        const float fk = __shfl_sync(FULL_MASK, f, min(k, n) - 1);
        const float edge = fk - (2.f * tau_s + 0x1p-22f * fabsf(fk));  // what may belong before the k-th
        if (!look && k < 32 && (__ballot_sync(FULL_MASK, close) >> k & 1u)) {
            // the last one in and the first one out are the same values: anything else as near?
            const float xk = __shfl_sync(FULL_MASK, px, k), bk = __shfl_sync(FULL_MASK, pb, k);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float fi = unordered(key[i]);
                if (key[i] != 0u && fi <= fk && fi >= edge && !(x[i] == xk && bias[i] == bk)) look = true;
            }
            look = __any_sync(FULL_MASK, look);
        } else if (!look && k == 32 && n == 32) {  // (no lane is left for the first one out)
            const uint32_t top = warp_max(mine);
            look = top != 0u && unordered(top) >= edge;
        }
        if (look) {
            // candidates: all from the edge on
            bool full = false;
            while (true) {
                const uint32_t top = warp_max(mine);
                if (top == 0u || !(unordered(top) >= edge)) break;
                if (n == 32) {
                    full = true;
                    break;
                }
                next_pick();
            }
            row64();
            if (!full) {
                pick = lane < n ? expert() : -1;
                double d = -INFINITY;
                if (pick >= 0) d = score64(a, logit_at<DT>(row, pick), m64, total64) + (double)a.bias[pick];
                int rank = 0;
                for (int j = 0; j < n; ++j) {
                    const double o = __shfl_sync(FULL_MASK, d, j);
                    const int oi = __shfl_sync(FULL_MASK, pick, j);
                    rank += o > d || (o == d && oi < pick);
                }
                // lane `rank` takes it
                int src = lane;
                for (int j = 0; j < n; ++j)
                    if (__shfl_sync(FULL_MASK, rank, j) == lane && lane < n) src = j;
                pick = __shfl_sync(FULL_MASK, pick, src);
            } else {
                // more than 32 candidates: every key of the row in 64 bits, k passes over them
                double d[NV];
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    d[i] = key[i] == 0u ? -INFINITY : score64(a, x[i], m64, total64) + (double)bias[i];
                pick = -1;
                for (int j = 0; j < k; ++j) {
                    double bd = -INFINITY;
                    int bi = 0x7fffffff;
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (d[i] > bd) bd = d[i], bi = e0 + i;
#pragma unroll
                    for (int o = 16; o; o >>= 1) {
                        const double od = __shfl_xor_sync(FULL_MASK, bd, o);
                        const int oi = __shfl_xor_sync(FULL_MASK, bi, o);
                        if (od > bd || (od == bd && oi < bi)) bd = od, bi = oi;
                    }
                    if (lane == j) pick = bi;
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (e0 + i == bi) d[i] = -INFINITY;
                }
            }
            px = pick >= 0 ? logit_at<DT>(row, pick) : 0.f;
        }
    }
    const bool here = lane < k && pick >= 0;
    const bool short_row = __any_sync(FULL_MASK, lane < k && pick < 0);

    // weights from the scores: with renormalisation relative to the largest
    // chosen logit, so that no sum of the k is zero
    float w = 0.f;
    float ref = m;
    if (a.renorm) ref = unordered(warp_max(here ? ordered(px) : 0u));
    if (softmax) {
        w = here ? expf(px - ref) : 0.f;
        if (!a.renorm) w /= total;
    } else if (here) {
        const float shift = a.renorm ? fminf(ref, 0.f) : 0.f;
        w = expf(fminf(px, 0.f) - shift) / (1.f + expf(-fabsf(px)));
    }
    if (a.renorm) w = w / warp_sum(w);
    if (lane < k) {
        a.ids[t * k + lane] = here ? pick : -1;
        a.w[t * k + lane] = here ? a.scale * w : 0.f;
    }
    if (short_row && lane == 0) atomicOr(a.err, MOE_DEVERR_LOGIT);
}

// A warp a row: any number of experts, few rows.
template <int NV, int DT>
__global__ void __launch_bounds__(rg_warps(NV) * 32) router_grouped_kernel(const __grid_constant__ RouterGroupedArgs a) {
    constexpr int WARPS = rg_warps(NV);
    __shared__ uint32_t sm_key[WARPS][NV * 32];
    __shared__ uint32_t sm_list[WARPS][32 * (NV + 1)];
    const int lane = threadIdx.x & 31, warp = warp_index();
    sm_list[warp][lane * (NV + 1) + NV] = 0u;
    after_previous();
    const RowPlan<NV> plan(a);
    for (int64_t t = (int64_t)blockIdx.x * WARPS + warp; t < a.T; t += (int64_t)gridDim.x * WARPS)
        route_row<NV, DT>(a, t, plan, sm_key[warp], sm_list[warp]);
}

// The same for the rows that the next kernel leaves (rare: not worth its registers).
template <int DT>
__device__ __noinline__ void route_row_again(const RouterGroupedArgs& a, int64_t t, uint32_t* sk, uint32_t* lists) {
    __syncwarp();
    lists[(threadIdx.x & 31) * 9 + 8] = 0u;
    route_row<8, DT>(a, t, RowPlan<8>(a), sk, lists);
    __syncwarp();
}

// Eight lanes a row, four rows a warp: up to 256 experts, whole lanes of
// groups, k <= 8.  What a whole warp spends on the picks of one row (a maximum
// over the lanes, whose it is, the next of its list), eight lanes do for four
// rows at once; a lane holds NE consecutive logits, as sorted lists of eight.
// Logits come by asynchronous copies, the next rows' while these are routed.
// Rows in which two keys or groups that may matter lie closer than FP32 tells
// apart, with fewer than k experts or with a sum of scores that is not finite
// are left to route_row.
// (65536 rows of 256, 8 groups: 55 us; a warp a row took 107, of 1077 instructions.)
constexpr int RO_WARPS = 4;
constexpr int RO_LIST(int ne) { return ne + 4; }  // words of a lane's lists, an odd number of 16-byte columns
template <int NE, int DT>
struct OctetBuffers {
    static constexpr int ES = DT == MOE_F32 ? 4 : 2;
    static constexpr int PITCH = NE * ES + 16;  // bytes of a lane's logits, an odd number of 16-byte columns
    alignas(16) uint8_t logits[32 * PITCH];
    alignas(16) uint32_t lists[32 * RO_LIST(NE)];
    alignas(16) uint32_t keys[32 * RO_LIST(NE)];
    static_assert(32 * RO_LIST(NE) >= 32 * 9, "route_row_again's lists");
};
template <int NE, int DT>
__global__ void __launch_bounds__(RO_WARPS * 32, NE == 32 ? 4 : 6) router_octets_kernel(const __grid_constant__ RouterGroupedArgs a) {
    using Buffers = OctetBuffers<NE, DT>;
    constexpr int ES = Buffers::ES, NS = NE / 8, LP = RO_LIST(NE);
    extern __shared__ __align__(16) uint8_t ro_smem[];
    const int lane = threadIdx.x & 31, warp = warp_index();
    Buffers& buf = reinterpret_cast<Buffers*>(ro_smem)[warp];
    const int sub = lane & 7, tk = lane >> 3, lane0 = lane & 24;
    const int E = a.E, k = a.k, per = E / 8, e0 = sub * per;
    const bool softmax = a.score == MOE_ROUTER_SOFTMAX, narrow = a.top_groups < a.groups;
    const bool top2 = a.group_score == MOE_ROUTER_GROUP_TOP2;
    const int q = 8 / a.groups;  // lanes of a group
    after_previous();

    const int64_t step = (int64_t)gridDim.x * RO_WARPS * 4;
    auto fetch = [&](int64_t t0) {  // chunk c of a row is lane c's
        const int64_t t = t0 + tk;
        if (t < a.T && sub * 16 < per * ES) {
            const uint8_t* from = static_cast<const uint8_t*>(a.logits) + t * a.stride * ES + sub * 16;
            uint8_t* to = buf.logits + lane0 * Buffers::PITCH + sub * 16;
#pragma unroll
            for (int c = 0; c < 8; ++c) cp_async_16_zfill(to + c * Buffers::PITCH, from + c * per * ES, 16);
        }
        cp_async_commit();
    };
    int64_t t0 = ((int64_t)blockIdx.x * RO_WARPS + warp) * 4;
    fetch(t0);

    float bias[NE];
    bool same_bias = true;
    {
        const float b0 = a.bias ? a.bias[0] : 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            bias[i] = !a.bias ? 0.f : i < per ? a.bias[e0 + i] : 0.f;
            if (i < per && bias[i] != b0) same_bias = false;
            bias[i] = fmaxf(bias[i], -INFINITY);  // (of NaN: -inf, absent)
        }
        same_bias = __all_sync(FULL_MASK, same_bias) && fabsf(b0) < INFINITY;
    }
    const bool by_logit = same_bias && !top2;

    for (; t0 < a.T; t0 += step) {
        const int64_t t = t0 + tk;
        float x[NE];
        cp_async_wait<0>();
        __syncwarp();
        {
            const uint8_t* const from = buf.logits + lane * Buffers::PITCH;
#pragma unroll
            for (int i = 0; i < NE; i += 4) {
                uint32_t w[4] = {0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u};
                if (i < per && t < a.T) {
                    if (DT == MOE_F32) {
                        const uint4 v = *reinterpret_cast<const uint4*>(from + i * ES);
                        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(from + i * ES);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t h = (e < 2 ? v.x : v.y) >> (e & 1) * 16 & 0xffffu;
                            w[e] = DT == MOE_BF16 ? h << 16 : __float_as_uint(__half2float(__ushort_as_half((uint16_t)h)));
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i + e] = fmaxf(__uint_as_float(w[e]), -INFINITY);
            }
        }
        __syncwarp();
        fetch(t0 + step);

        // scores and keys, as in route_row; keys stay floats, -inf for absent
        float m = 0.f, total = 1.f;
        if (softmax && (!same_bias || (narrow && top2) || !a.renorm)) {
            m = x[0];
#pragma unroll
            for (int i = 1; i < NE; ++i) m = fmaxf(m, x[i]);
#pragma unroll
            for (int o = 1; o < 8; o *= 2) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, o));
            total = 0.f;
#pragma unroll
            for (int i = 0; i < NE; ++i) total += exp2_ftz((x[i] - m) * 1.44269504f);
#pragma unroll
            for (int o = 1; o < 8; o *= 2) total += __shfl_xor_sync(FULL_MASK, total, o);
        }
        const float inv = 1.f / total, tau_s = score_error(softmax, total);
        float best = -INFINITY, second = -INFINITY;
        auto see = [&](float v) {
            second = fmaxf(second, fminf(best, v));
            best = fmaxf(best, v);
        };
        if (!same_bias) {
            if (softmax)
#pragma unroll
                for (int i = 0; i < NE; ++i)
                    x[i] = x[i] > -INFINITY ? fmaf(exp2_ftz((x[i] - m) * 1.44269504f), inv, bias[i]) : -INFINITY;
            else
#pragma unroll
                for (int i = 0; i < NE; ++i)
                    x[i] = x[i] > -INFINITY ? rcp_fast(1.f + exp2_ftz(x[i] * -1.44269504f)) + bias[i] : -INFINITY;
        } else if (narrow && top2) {  // (the order is the logits', a group's worth is of scores)
#pragma unroll
            for (int i = 0; i < NE; ++i)
                see(x[i] == -INFINITY ? -INFINITY
                    : softmax         ? exp2_ftz((x[i] - m) * 1.44269504f) * inv
                                      : rcp_fast(1.f + exp2_ftz(x[i] * -1.44269504f)));
        }
        if (narrow && (!same_bias || !top2))
#pragma unroll
            for (int i = 0; i < NE; ++i) see(x[i]);
        // this row is left to route_row; a sum of NaN (a logit of +inf) leaves no key that could be compared
        bool again = !(total < INFINITY);
        if (narrow) {
            for (int o = 1; o < q; o *= 2) {
                const float b2 = __shfl_xor_sync(FULL_MASK, best, o), s2 = __shfl_xor_sync(FULL_MASK, second, o);
                second = fmaxf(fmaxf(second, s2), fminf(best, b2));
                best = fmaxf(best, b2);
            }
            float worth = top2 ? best + second : best;
            if (!(worth >= -INFINITY)) worth = -INFINITY;
            int rank = 0;
            for (int g = 0; g < 8; g += q) {
                const float o = __shfl_sync(FULL_MASK, worth, lane0 + g);
                const bool other = g != (sub & -q);
                rank += other && (o > worth || (o == worth && g < sub));
            }
            if (!by_logit) {  // the border between the last group in and the first one out
                const float err = worth_error(worth, best, top2 ? second : 0.f, tau_s);
                float last = rank < a.top_groups ? worth - err : INFINITY, next = rank < a.top_groups ? -INFINITY : worth + err;
#pragma unroll
                for (int o = 1; o < 8; o *= 2) {
                    last = fminf(last, __shfl_xor_sync(FULL_MASK, last, o));
                    next = fmaxf(next, __shfl_xor_sync(FULL_MASK, next, o));
                }
                again |= last <= next && next > -INFINITY && last < INFINITY;
            }
            if (rank >= a.top_groups)
#pragma unroll
                for (int i = 0; i < NE; ++i) x[i] = -INFINITY;
        }

        // lists of eight
        float* const lists = reinterpret_cast<float*>(buf.lists);
        float* const keys = reinterpret_cast<float*>(buf.keys);
        float head[NS];
#pragma unroll
        for (int l = 0; l < NS; ++l) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = x[l * 8 + i];
            *reinterpret_cast<float4*>(keys + lane * LP + l * 8) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(keys + lane * LP + l * 8 + 4) = make_float4(v[4], v[5], v[6], v[7]);
            sort_down(v);
            head[l] = v[0];
            *reinterpret_cast<float4*>(lists + lane * LP + l * 8) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(lists + lane * LP + l * 8 + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
        __syncwarp();
        float pick_key = -INFINITY, beyond = -INFINITY;
        uint32_t taken = 0u;  // a byte for each list
        int from = 0, which = 0;
        const int want = same_bias ? k : k + 1;
#pragma unroll 1
        for (int j = 0; j < want; ++j) {
            float mine = head[0];
#pragma unroll
            for (int l = 1; l < NS; ++l) mine = fmaxf(mine, head[l]);
            float top = mine;
#pragma unroll
            for (int o = 1; o < 8; o *= 2) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
            const uint32_t has = __ballot_sync(FULL_MASK, mine == top) >> lane0 & 0xffu;
            const int owner = __ffs(has | 0x80u) - 1;  // (none has a maximum of NaN: any lane, the row is done again)
            int l = NS - 1;
#pragma unroll
            for (int i = NS - 2; i >= 0; --i)
                if (head[i] == top) l = i;
            const int of = __shfl_sync(FULL_MASK, l, lane0 + owner);
            if (sub == owner) {
                const uint32_t at = (taken >> 8 * l & 0xffu) + 1u;
                taken += 1u << 8 * l;
                const float next = at < 8u ? lists[lane * LP + l * 8 + at] : -INFINITY;
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    if (i == l) head[i] = next;
            }
            if (sub == j) pick_key = top, from = lane0 + owner, which = of;
            if (j == k) beyond = top;
        }
        const bool mine = sub < k;
        again |= mine && !(pick_key > -INFINITY);  // fewer than k experts
        // which of the list's eight experts: equal keys come in their order
        int skip = 0;
        {
            const float key_before = __shfl_up_sync(FULL_MASK, pick_key, 1, 8);
            const int list_before = __shfl_up_sync(FULL_MASK, from * 8 + which, 1, 8);
            const bool twin = sub > 0 && mine && key_before == pick_key && list_before == from * 8 + which;
            if (__any_sync(FULL_MASK, twin))
                for (int i = 1; i < 8; ++i) {
                    const int before = __shfl_up_sync(FULL_MASK, skip, 1, 8);
                    skip = twin ? before + 1 : 0;
                }
        }
        int pick = 0;
        {
            const float4 lo = *reinterpret_cast<const float4*>(keys + from * LP + which * 8);
            const float4 hi = *reinterpret_cast<const float4*>(keys + from * LP + which * 8 + 4);
            const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            int at = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (v[i] == pick_key && skip-- == 0) at = i;
            pick = (from & 7) * per + which * 8 + at;
        }
        if (!same_bias) {
            float after = __shfl_down_sync(FULL_MASK, pick_key, 1, 8);
            if (sub == k - 1) after = beyond;
            const float gap = pick_key - after;  // (infinite: no key is left behind this one)
            again |= mine && gap < INFINITY && gap <= 2.f * tau_s + 0x1p-22f * fmaxf(fabsf(pick_key), fabsf(after));
        }
        // weights, as in route_row (all lanes take part in the exchanges)
        {
            const bool there = mine && t < a.T && pick_key > -INFINITY;
            const void* const row = static_cast<const uint8_t*>(a.logits) + t * a.stride * ES;
            const float px = there ? logit_at<DT>(row, pick) : -INFINITY;
            float ref = m, w = 0.f;
            if (a.renorm) {
                ref = px;
#pragma unroll
                for (int o = 1; o < 8; o *= 2) ref = fmaxf(ref, __shfl_xor_sync(FULL_MASK, ref, o));
            }
            if (softmax) {
                w = there ? expf(px - ref) : 0.f;
                if (!a.renorm) w /= total;
            } else if (there) {
                const float shift = a.renorm ? fminf(ref, 0.f) : 0.f;
                w = expf(fminf(px, 0.f) - shift) / (1.f + expf(-fabsf(px)));
            }
            float sum = w;
            if (a.renorm) {
#pragma unroll
                for (int o = 1; o < 8; o *= 2) sum += __shfl_xor_sync(FULL_MASK, sum, o);
                w /= sum;
            }
            again = __ballot_sync(FULL_MASK, again) >> lane0 & 0xffu;
            if (there && !again) {
                a.ids[t * k + sub] = pick;
                a.w[t * k + sub] = a.scale * w;
            }
        }
        // (rows of the warp that are left: all lanes go there together)
        for (uint32_t left = __ballot_sync(FULL_MASK, again && sub == 0 && t < a.T); left; left &= left - 1u)
            route_row_again<DT>(a, t0 + ((__ffs(left) - 1) >> 3), buf.keys, buf.lists);
    }
    cp_async_wait<0>();
}

template <int NV, int DT>
static cudaError_t launch_rg(const RouterGroupedArgs& a, const DeviceInfo& di, cudaStream_t st) {
    constexpr int WARPS = rg_warps(NV);
    const int64_t blocks = (a.T + WARPS - 1) / WARPS;
    return launch_after(router_grouped_kernel<NV, DT>, dim3((unsigned)std::min<int64_t>(blocks, di.sm_count * 8)), WARPS * 32,
                        0, st, a);
}

template <int NE, int DT>
static cudaError_t launch_ro(const RouterGroupedArgs& a, const DeviceInfo& di, cudaStream_t st) {
    constexpr size_t smem = RO_WARPS * sizeof(OctetBuffers<NE, DT>);
    static SmemOnce once;
    const cudaError_t e = once.set(reinterpret_cast<const void*>(router_octets_kernel<NE, DT>), (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (a.T + RO_WARPS * 4 - 1) / (RO_WARPS * 4);
    return launch_after(router_octets_kernel<NE, DT>, dim3((unsigned)std::min<int64_t>(blocks, di.sm_count * (NE == 32 ? 4 : 6))),
                        RO_WARPS * 32, smem, st, a);
}

// Eight lanes a row where there are rows for all SMs' warps (see its comment
// for the shapes): below that a whole warp is sooner done with its row.
static bool octets_fit(const RouterGroupedArgs& a, int dtype, const DeviceInfo& di) {
    const int es = dtype == MOE_F32 ? 4 : 2;
    return a.T >= di.sm_count * 32 && a.E <= 256 && a.E * es % 128 == 0 && a.k <= 8 && 8 % a.groups == 0 &&
           a.stride * es % 16 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
}

template <int DT>
static cudaError_t launch_rg_dt(const RouterGroupedArgs& a, const DeviceInfo& di, cudaStream_t st) {
    if (octets_fit(a, DT, di)) {
        if (a.E <= 64) return launch_ro<8, DT>(a, di, st);
        if (a.E <= 128) return launch_ro<16, DT>(a, di, st);
        return launch_ro<32, DT>(a, di, st);
    }
    if (a.E <= 128) return launch_rg<4, DT>(a, di, st);
    if (a.E <= 256) return launch_rg<8, DT>(a, di, st);
    if (a.E <= 512) return launch_rg<16, DT>(a, di, st);
    return launch_rg<32, DT>(a, di, st);
}

cudaError_t launch_router_grouped(RouterGroupedArgs a, int dtype, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    a.err = di.err_word;
    const int64_t four = dtype == MOE_F32 ? 16 : 8;  // bytes
    a.vec = a.E % 4 == 0 && a.stride % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % four == 0;
    if (dtype == MOE_F32) return launch_rg_dt<MOE_F32>(a, di, st);
    return dtype == MOE_BF16 ? launch_rg_dt<MOE_BF16>(a, di, st) : launch_rg_dt<MOE_F16>(a, di, st);
}

}  // namespace moedec
