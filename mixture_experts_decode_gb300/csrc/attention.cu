// attention.cu -- attention of one new token per sequence over a paged
// key-value cache, with an optional sliding window and first tokens that stay
// visible, split evenly over the grid and joined inside the same launch.
//
// Mathematics.  For each sequence b and query head h (key-value head
// h / (Hq / Hkv)), over the visible keys j:
//   s_j = scale * q . k_j,   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
// in one pass: each warp keeps the running maximum m (base 2), sum l and
// unnormalised o, rescaling o only when m grows; warps, then pieces of a
// sequence, combine by exp2(m_piece - m) weights.  All of it is FP32.
//
// Bound: HBM, each visible K and V row once (2 * D * bytes per key and
// key-value head).  The query heads that share a key-value head are the N
// columns of the products, so a key row is read once for all of them:
//   S^T [16 keys x heads] = K [16 x D] * Q^T,   O^T [D x heads] += V^T * P^T
// with mma.m16n8k16: 8 heads fill one N tile exactly, and the score
// accumulator becomes the second product's B operand by one 8x8 transpose
// (movmatrix).  A tcgen05 product needs 64 or 128 rows in M and moves its
// accumulator through TMEM; here the products keep the tensor pipe busy for 27 %
// of the time (E4M3) or 12 % (BF16), so the warp-level instruction with its
// operands in registers is the shorter path.
//
// Rounding choices: scores, softmax and sums are FP32.  The second product
// takes 16-bit operands; p is given to it as hi + lo (two 16-bit values, an
// error near 2^-17 of p in BF16 and 2^-22 in FP16), because one 16-bit
// rounding of p would cost as much as rounding the output.  FP16 operands
// hold 2^14 p (at most 2^15), so that a long tail of keys far below the
// maximum is kept down to p = 2^-38; l carries the same factor.  E4M3 codes
// widen to FP16 exactly; a BF16 q then goes to FP16 after a power-of-two scaling of its head's row
// (the largest element in [2^9, 2^10]), exact for elements within 2^-23 of
// the row's largest, and smaller ones are off by less than FP32's own sum.
//
// Layout: every warp has its own ring of cp.async stages of 16 keys (K and V),
// so no barrier of the block sits in the main loop.  Work is counted in units
// of 64 visible keys of one (sequence, key-value head) item; each block takes
// an equal contiguous run of units (so ragged batches stay balanced), and the
// last block to finish an item that was cut joins its pieces in order, which
// keeps the result independent of timing.
//
// Measured: 4 sequences of 124000 keys, 64 / 8 heads of 128, E4M3 (1.02 GB):
// 176 to 194 us, 5.3 to 5.8 TB/s; 32 sequences of 0..32768, 32 / 4 heads of
// 128, BF16 (201 MB): 44 us, 4.5 TB/s; one of 777 keys: 10 us, latency alone.
#include "block_common.cuh"
#include "internal.h"

namespace moedec {

namespace {

constexpr int ATT_WARPS = 4;
constexpr int ATT_THREADS = ATT_WARPS * 32;
constexpr int ATT_STEP = 16;                     // keys per warp step
constexpr int ATT_UNIT = ATT_STEP * ATT_WARPS;   // keys per unit of work
// What beginning a piece costs, in units: filling the ring and combining the
// warps take as long as about two units of keys.
constexpr int ATT_BEGIN = 2;
// A block takes at least this much, one unit and its beginning: cutting finer
// only adds joins, and coarser lets a block do items one after the other
// (777 keys of one sequence: 13.0 us at 1, 10.1 at 3, 12.0 at 5).
constexpr int ATT_LEAST = 3;
// An item of at most so many units is not cut: its steps one after the other
// take less than a join (64 sequences of 200 keys: 10.0 us against 15.8; 11 of
// 122 visible keys, D = 256: 8.1 against 12.2).
constexpr int ATT_WHOLE = 4;
constexpr int KV_BF16 = 0, KV_F16 = 1, KV_E4M3 = 2;

// Blocks per SM that the registers are cut for, and stages per warp in their
// share of the 228 KB: three blocks of two stages of D = 128 BF16 beat two of
// three (the warps' fixed latencies, not the loads, are what is waited for).
constexpr int att_blocks(int dp, int nt) { return dp == 64 && nt == 1 ? 4 : dp == 256 || nt == 2 ? 2 : 3; }
constexpr int att_stages(int dp, int es, int nt) {
    const int s = (att_blocks(dp, nt) == 4 ? 49152 : att_blocks(dp, nt) == 3 ? 66000 : 98304) /
                  (ATT_WARPS * 2 * ATT_STEP * dp * es);
    const int least = es == 1 ? 3 : 2;  // (the sums of two N tiles take three E4M3 stages)
    return s < least ? least : (s > 6 ? 6 : s);
}

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (BF)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if (BF) return bf16x2_to_float2(v);
    __half2 h;
    memcpy(&h, &v, 4);
    return __half22float2(h);
}
// Two E4M3 codes in the low / high half of a word -> FP16 pair, exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{ .reg .b16 l, h;\n\t mov.b32 {l, h}, %2;\n\t cvt.rn.f16x2.e4m3x2 %0, l;\n\t cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.f : m; }

}  // namespace

// The visible keys of a sequence of n tokens, as one run 0 .. vis-1 that maps
// to tokens: the first `head` stand for tokens 0 .. head-1, the rest for
// tokens from head + skip on.
struct Visible {
    int vis, head, skip;
};
__device__ __forceinline__ Visible visible_keys(int n, int window, int sinks) {
    if (window == 0 || n <= window) return {n, n, 0};
    const int start = n - window;
    const int head = min(sinks, start);
    return {head + window, head, start - head};
}

__device__ __forceinline__ void add_scaled(float4& s, float f, const float4& v) {
    s.x += f * v.x, s.y += f * v.y, s.z += f * v.z, s.w += f * v.w;
}

// Four output values of a head from its joined sums; ml = (maximum, l).
// l = 0 (no visible key, or every score -inf) gives 0 and a log-sum of -inf.
template <bool QBF>
__device__ __forceinline__ void store_head4(const AttnArgs& a, int b, int h, int dim, const float4& sum, float2 ml,
                                            float shift) {
    const int64_t row = (int64_t)b * a.Hq + h;
    const float f = ml.y == 0.f ? 0.f : a.v_scale / ml.y;
    float v[4] = {sum.x * f, sum.y * f, sum.z * f, sum.w * f};
    uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.D + dim;
    const uint32_t lo = pack2<QBF>(v[0], v[1]), hi = pack2<QBF>(v[2], v[3]);
    if (a.out_aligned) {
        *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
    } else {
        out[0] = (uint16_t)lo, out[1] = (uint16_t)(lo >> 16);
        out[2] = (uint16_t)hi, out[3] = (uint16_t)(hi >> 16);
    }
    if (dim == 0 && a.lse) a.lse[row] = ml.y == 0.f ? -INFINITY : (ml.x - shift + log2f(ml.y)) * 0.693147180559945309f;
}

// Joins n pieces of an item, piece i at slot(i), in their order: the sums go
// to `put` four dims at a time with the joined (maximum, l).  Every thread
// joins its own dims with eight pieces' loads in flight at a time, the maxima
// and sums among them, so a join of eight is one round trip to L2.
constexpr int ATT_JOIN = 8;                                     // pieces of a group
constexpr int ATT_JOIN_MOST = ATTN_MAX_BLOCKS / ATT_JOIN + 1;   // groups of an item
template <class Slot, class Put>
__device__ __forceinline__ void join_slots(const AttnArgs& a, int n, int heads, Slot slot, Put put) {
    const float2* mls = reinterpret_cast<const float2*>(a.ws_ml);
    for (int e = threadIdx.x; e < heads * (a.D / 4); e += ATT_THREADS) {
        const int h = e / (a.D / 4), dim = (e - h * (a.D / 4)) * 4;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int p0 = 0; p0 < n; p0 += 8) {
            float4 v[8];
            float2 ml[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // beyond the end the last piece again, with weight 0
                const int64_t at = (int64_t)slot(min(p0 + i, n - 1)) * a.hpi + h;
                ml[i] = __ldcg(mls + at);
                v[i] = __ldcg(reinterpret_cast<const float4*>(a.ws_o + at * a.D + dim));
            }
            float mn = m;
#pragma unroll
            for (int i = 0; i < 8; ++i) mn = fmaxf(mn, ml[i].x);
            const float mu = finite_or_zero(mn);
            const float old = exp2_fast(m - mu);
            m = mn;
            l *= old;
            sum.x *= old, sum.y *= old, sum.z *= old, sum.w *= old;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (p0 + i < n) {
                    const float f = exp2_fast(ml[i].x - mu);
                    l += f * ml[i].y;
                    add_scaled(sum, f, v[i]);
                }
        }
        put(h, dim, sum, make_float2(m, l));
    }
}

// True in every thread of the block that is the last of `n` to arrive at the
// counter, which is then zero again.  What the blocks wrote before is visible
// to it.  (A counter that began above zero is noticed only where some block
// finds n or more: a lower value looks like an arrival.)
__device__ __forceinline__ bool arrive_last(int* counter, int n, int* err, int* flag) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int old = atomicAdd(counter, 1);
        if (old < 0 || old >= n) atomicOr(err, MOE_DEVERR_WORKSPACE);
        if (old == n - 1) *counter = 0;
        __threadfence();
        *flag = old == n - 1;
    }
    __syncthreads();
    return *flag != 0;
}

// The pieces of an item cut over blocks c1 .. c2 (this block's is written):
// the last block of each eight joins theirs into the first one's place, the
// last of those joins the groups (one level where eight blocks suffice), so
// no block reads more than 81 pieces.  Counters: an item's first group by c1
// (no other item begins in that block and goes on), its later groups and the
// item itself by block / 8 (an item of more than eight blocks is the only one
// with a later group, or an end, in such a place).
template <bool QBF>
__device__ __noinline__ void join_pieces(const AttnArgs& a, int c1, int c2, int b, int head0, int heads, float shift,
                                         float2* head_ml, int* flag) {
    const int pieces = c2 - c1 + 1;
    const int grp = ((int)blockIdx.x - c1) / ATT_JOIN;
    const int g0 = c1 + grp * ATT_JOIN;
    const int in_group = min(ATT_JOIN, pieces - grp * ATT_JOIN);
    int* const later = a.counters + ATTN_MAX_BLOCKS;
    int* const ends = later + ATT_JOIN_MOST;
    auto slot = [&](int c) { return 2 * c + (c == c1 ? 1 : 0); };
    auto finish = [&](int h, int dim, const float4& sum, float2 ml) { store_head4<QBF>(a, b, head0 + h, dim, sum, ml, shift); };
    if (!arrive_last(grp == 0 ? a.counters + c1 : later + g0 / ATT_JOIN, in_group, a.err, flag)) return;
    if (pieces <= ATT_JOIN) {
        join_slots(a, pieces, heads, [&](int p) { return slot(c1 + p); }, finish);
        return;
    }
    // The group takes its first piece's place: each thread has read its own
    // dims of it by then, and the maxima and sums, which all threads read, are
    // put there after a barrier.
    const int64_t to = (int64_t)slot(g0) * a.hpi;
    join_slots(a, in_group, heads, [&](int p) { return slot(g0 + p); }, [&](int h, int dim, const float4& sum, float2 ml) {
        *reinterpret_cast<float4*>(a.ws_o + (to + h) * a.D + dim) = sum;
        if (dim == 0) head_ml[h] = ml;
    });
    __syncthreads();
    if ((int)threadIdx.x < heads) reinterpret_cast<float2*>(a.ws_ml)[to + threadIdx.x] = head_ml[threadIdx.x];
    const int groups = (pieces + ATT_JOIN - 1) / ATT_JOIN;
    if (!arrive_last(ends + c1 / ATT_JOIN, groups, a.err, flag)) return;
    join_slots(a, groups, heads, [&](int p) { return slot(c1 + p * ATT_JOIN); }, finish);
}

template <int DP, int NT, int KV, bool QBF>
__global__ void __launch_bounds__(ATT_THREADS, att_blocks(DP, NT)) paged_attention_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int ES = KV == KV_E4M3 ? 1 : 2;
    constexpr bool BF = KV == KV_BF16;  // operand type of the products
    constexpr int ROW = DP * ES;        // bytes of a key's row in shared memory
    constexpr int CHP = ROW / 16;
    constexpr int NST = att_stages(DP, ES, NT);
    constexpr int HALF = ATT_STEP * ROW;  // bytes of K (or V) in a stage
    constexpr int NK = DP / 16;
    constexpr int NH = NT * 8;
    constexpr float P_SHIFT = BF ? 0.f : 14.f;
    constexpr float SLACK = BF ? 8.f : 1.f;  // FP16 holds 2^15 p
    constexpr int SO = DP + 4;               // floats of a head's row of o in shared memory

    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_index();
    const int g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + (size_t)warp * NST * 2 * HALF;
    uint8_t* tail = smem + (size_t)ATT_WARPS * NST * 2 * HALF;
    uint32_t* live = reinterpret_cast<uint32_t*>(tail) + warp * NST;  // readable keys of each stage
    float* sm_m = reinterpret_cast<float*>(tail + ATT_WARPS * NST * 4);  // [warps][NH]
    float* sm_l = sm_m + ATT_WARPS * NH;
    float2* head_ml = reinterpret_cast<float2*>(sm_l + ATT_WARPS * NH);      // [NH]
    int64_t* sm_warp = reinterpret_cast<int64_t*>(head_ml + NH);            // [warps] + carry
    int64_t* prefix = sm_warp + 8;                                          // [B] cost up to and with b

    after_previous();
    const int nk = a.D / 16;
    const int chunks16 = a.D * ES / 16;
    const int64_t cap = (int64_t)a.max_pages * a.page;

    // cost of an item of each sequence, scanned over the batch
    int64_t carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += ATT_THREADS) {
        const int b = b0 + tid;
        int64_t u = 0;
        if (b < a.B) {
            const int n = a.lens[b];
            if (n < 0 || n > cap) {
                if (blockIdx.x == 0) atomicOr(a.err, MOE_DEVERR_PAGE);
            }
            const int nn = (int)(n < 0 ? 0 : (n > cap ? cap : n));
            const Visible v = visible_keys(nn, a.window, a.sinks);
            u = ((int64_t)v.vis + ATT_UNIT - 1) / ATT_UNIT;
            if (u) u += ATT_BEGIN;
        }
        int64_t s = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(FULL_MASK, s, o);
            if (lane >= o) s += v;
        }
        if (lane == 31) sm_warp[warp] = s;
        __syncthreads();
        for (int w = 0; w < warp; ++w) s += sm_warp[w];
        if (b < a.B) prefix[b] = s + carry;
        if (tid == ATT_THREADS - 1) sm_warp[ATT_WARPS] = s;
        __syncthreads();
        carry += sm_warp[ATT_WARPS];
    }
    // a sequence without keys has no units: its rows are written here
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
        if (prefix[b] == (b ? prefix[b - 1] : 0)) {
            for (int i = tid; i < a.Hq * a.D; i += ATT_THREADS)
                static_cast<uint16_t*>(a.out)[(int64_t)b * a.Hq * a.D + i] = 0;
            if (a.lse)
                for (int h = tid; h < a.Hq; h += ATT_THREADS) a.lse[(int64_t)b * a.Hq + h] = -INFINITY;
        }
    const int items = a.Hkv * a.chunks;  // items of one sequence
    const int64_t total = carry * items;
    const int64_t blocks = min((int64_t)gridDim.x, (total + ATT_LEAST - 1) / ATT_LEAST);
    if ((int64_t)blockIdx.x >= blocks) return;
    // Block c takes the costs [total c / blocks, total (c + 1) / blocks), but
    // an item is not cut within the cost of beginning it, and a short one not
    // at all: a border there moves to the item's start.
    int64_t u = total * blockIdx.x / blocks;
    const int64_t u_end = total * (blockIdx.x + 1) / blocks;
    int b = 0;
    {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] * items > u)
                hi = mid;
            else
                lo = mid + 1;
        }
        b = lo;
    }

    while (u < u_end) {
        while (prefix[b] * items <= u) ++b;
        const int64_t before = b ? prefix[b - 1] : 0;
        const int64_t cost = prefix[b] - before;
        const int64_t rel = u - before * items;
        const int item = (int)(rel / cost);
        const int64_t first_u = before * items + (int64_t)item * cost;
        const int64_t units = cost - ATT_BEGIN;
        if (u_end - first_u <= (units <= ATT_WHOLE ? cost - 1 : ATT_BEGIN)) break;  // it begins in the next block
        const int64_t t0 = units <= ATT_WHOLE ? 0 : max((int64_t)0, u - first_u - ATT_BEGIN);
        const int64_t t1 = min(units, u_end - first_u - ATT_BEGIN);
        const int kvh = item / a.chunks, chunk = item - kvh * a.chunks;
        const int head0 = kvh * a.G + chunk * a.hpi;
        const int heads = min(a.hpi, a.G - chunk * a.hpi);
        const int n_raw = a.lens[b];
        const int n = (int)(n_raw > cap ? cap : n_raw);
        const Visible vis = visible_keys(n, a.window, a.sinks);
        const int key_end = (int)min((int64_t)vis.vis, t1 * ATT_UNIT);
        const int step0 = (int)(t0 * ATT_WARPS) + warp;
        const int64_t step_end = ((int64_t)key_end + ATT_STEP - 1) / ATT_STEP;
        const int steps = step0 < step_end ? (int)((step_end - step0 + ATT_WARPS - 1) / ATT_WARPS) : 0;
        const int32_t* table = a.table + (int64_t)b * a.table_stride;
        const uint8_t* kbase = static_cast<const uint8_t*>(a.k) + (int64_t)kvh * a.k_sh * ES;
        const uint8_t* vbase = static_cast<const uint8_t*>(a.v) + (int64_t)kvh * a.v_sh * ES;

        // Nothing from here to the sums' end branches per lane, because the
        // matrix instructions need the whole warp together.
        // Lanes 0..15 find the row of one key each in the K cache, lanes 16..31
        // the same keys' in the V cache, one step ahead of its use; beyond the
        // last key they look the last one up again and drop it.
        int pg = 0, off = 0;
        bool in_range = false;
        auto find = [&](int i) {
            if (i >= steps) return;
            const uint32_t key0 = (uint32_t)(step0 + i * ATT_WARPS) * ATT_STEP + (lane & 15);
            const int key = (int)min(key0, (uint32_t)key_end - 1u);
            const int tok = key < vis.head ? key : key + vis.skip;
            const int pi = (int)(((uint64_t)(uint32_t)tok * a.page_mul) >> a.page_shift);
            off = tok - pi * a.page;
            in_range = key0 < (uint32_t)key_end;
            pg = table[pi];  // (used by the next issue)
        };
        constexpr int ROWS = 32 / CHP;  // rows that the warp copies at once
        const int col = lane % CHP, row0 = lane / CHP;
        const uint8_t* kcol = kbase + (col < chunks16 ? col * 16 : 0);
        const uint8_t* vcol = vbase + (col < chunks16 ? col * 16 : 0);
        auto issue = [&](int i, int st) {
            if (i < steps) {
                const bool known = pg >= 0 && pg < a.num_pages;
                if (__any_sync(FULL_MASK, !known)) atomicOr(a.err, known ? 0 : MOE_DEVERR_PAGE);
                const bool have = known && in_range;
                const int64_t row_at =  // bytes from the head's first row
                    have ? (pg * (lane < 16 ? a.k_sp : a.v_sp) + off * (lane < 16 ? a.k_st : a.v_st)) * ES : 0;
                const uint32_t mask = __ballot_sync(FULL_MASK, have) & 0xffffu;
                live[st] = mask;
                const uint32_t copied = col < chunks16 ? mask : 0u;  // 0 bytes write zeros
                uint8_t* sk = ring + st * 2 * HALF;
#pragma unroll
                for (int it = 0; it < ATT_STEP / ROWS; ++it) {
                    const int row = it * ROWS + row0;
                    const int64_t ka = __shfl_sync(FULL_MASK, row_at, row), va = __shfl_sync(FULL_MASK, row_at, row + 16);
                    const int bytes = (copied >> row & 1u) << 4;
                    const int ck = KV == KV_E4M3 ? (CHP >= 8 ? col ^ ((row & 1) << 2) : col) : col ^ (row & 7);
                    const int cv = KV == KV_E4M3 ? (CHP >= 8 ? col ^ (((row >> 1) & 3) << 1) : col ^ (((row >> 1) & 1) << 1))
                                                 : col ^ (row & 7);
                    cp_async_16_zfill(sk + row * ROW + ck * 16, kcol + ka, bytes);
                    cp_async_16_zfill(sk + HALF + row * ROW + cv * 16, vcol + va, bytes);
                }
            }
            cp_async_commit();
        };
        find(0);
#pragma unroll 1
        for (int i = 0; i < NST - 1; ++i) {
            issue(i, i);
            find(i + 1);
        }

        // q as the first product's B operand (column = head g of the tile)
        uint32_t qf[NT][NK][2];
        float sl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = nt * 8 + g;
            const uint16_t* qrow =
                static_cast<const uint16_t*>(a.q) + (int64_t)b * a.q_sb + (int64_t)(head0 + (h < heads ? h : 0)) * a.q_sh;
            if (KV != KV_E4M3) {
#pragma unroll
                for (int kk = 0; kk < NK; ++kk) {
                    const bool on = h < heads && kk < nk;
                    qf[nt][kk][0] = on ? *reinterpret_cast<const uint32_t*>(qrow + kk * 16 + 2 * t) : 0u;
                    qf[nt][kk][1] = on ? *reinterpret_cast<const uint32_t*>(qrow + kk * 16 + 2 * t + 8) : 0u;
                }
                sl[nt][0] = sl[nt][1] = a.scale_log2;
            } else {
                // the thread's 16 codes of a key are dims 64j + 16t ..; product i
                // of the block takes four of them
                float amax = 0.f;
#pragma unroll
                for (int kk = 0; kk < NK; ++kk) {
                    const int dim = (kk >> 2) * 64 + t * 16 + (kk & 3) * 4;
                    const bool on = h < heads && dim < a.D;
                    uint2 v = on ? *reinterpret_cast<const uint2*>(qrow + dim) : make_uint2(0u, 0u);
                    qf[nt][kk][0] = v.x;
                    qf[nt][kk][1] = v.y;
                    if (QBF) {
                        const float2 p = bf16x2_to_float2(v.x), r = bf16x2_to_float2(v.y);
                        amax = fmaxf(fmaxf(amax, fmaxf(fabsf(p.x), fabsf(p.y))), fmaxf(fabsf(r.x), fabsf(r.y)));
                    }
                }
                float back = 1.f;
                if (QBF) {
                    amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, 2));
                    // 2^e <= amax < 2^(e+1); q * 2^(9-e), undone in the scale
                    int e = (int)(__float_as_uint(amax) >> 23) - 127;
                    e = max(-100, min(e, 127));
                    const float fwd = __uint_as_float((uint32_t)(127 + min(9 - e, 109)) << 23);
                    back = __uint_as_float((uint32_t)(127 - min(9 - e, 109)) << 23);
#pragma unroll
                    for (int kk = 0; kk < NK; ++kk)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float2 p = bf16x2_to_float2(qf[nt][kk][r]);
                            qf[nt][kk][r] = pack2<false>(p.x * fwd, p.y * fwd);
                        }
                }
                sl[nt][0] = a.scale_log2 * __shfl_sync(FULL_MASK, back, 8 * t);
                sl[nt][1] = a.scale_log2 * __shfl_sync(FULL_MASK, back, 8 * t + 4);
            }
        }

        float o[NK][NT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int kk = 0; kk < NK; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[kk][nt][i] = 0.f;
        }

        int use = 0;  // stage of step i
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
            cp_async_wait<NST - 2>();
            __syncwarp();
            issue(i + NST - 1, use == 0 ? NST - 1 : use - 1);  // into the stage that step i - 1 has left
            find(i + NST);
            const uint8_t* sk = ring + use * 2 * HALF;
            const uint8_t* sv = sk + HALF;
            const uint32_t mask = live[use];
            if (++use == NST) use = 0;

            float s[NT][4];
            {
                float s2[NT][2][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s2[nt][0][j] = s2[nt][1][j] = 0.f;
                if (KV != KV_E4M3) {
                    const int row = lane & 15;
                    const uint32_t base = smem_addr(sk + row * ROW);
#pragma unroll
                    for (int kk = 0; kk < NK; ++kk)
                        if (kk < nk) {
                            uint32_t k4[4];
                            ldsm_x4(k4, base + (((kk * 2 + (lane >> 4)) ^ (row & 7)) << 4));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816<BF>(s2[nt][kk & 1], k4, qf[nt][kk][0], qf[nt][kk][1]);
                        }
                } else {
#pragma unroll
                    for (int j = 0; j < (DP + 63) / 64; ++j) {
                        const int col = j * 4 + t;
                        const int sw = CHP >= 8 ? col ^ ((g & 1) << 2) : col;
                        const uint4 lo = *reinterpret_cast<const uint4*>(sk + g * ROW + sw * 16);
                        const uint4 hi = *reinterpret_cast<const uint4*>(sk + (g + 8) * ROW + sw * 16);
                        const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t k4[4];
                            e4m3x4_to_f16(wl[q], k4[0], k4[2]);
                            e4m3x4_to_f16(wh[q], k4[1], k4[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<false>(s2[nt][q & 1], k4, qf[nt][j * 4 + q][0], qf[nt][j * 4 + q][1]);
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool on = (mask >> (g + (j >> 1) * 8)) & 1u;
                        s[nt][j] = on ? (s2[nt][0][j] + s2[nt][1][j]) * sl[nt][j & 1] : -INFINITY;
                    }
            }

            // The reference m of the exponents only has to stay near the running
            // maximum: it moves, and o and l with it, when some score passes it
            // by more than SLACK (p <= 2^SLACK), which is rare after the first
            // steps and spares the other steps the reduction over the keys.
            bool grew = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) grew |= fmaxf(s[nt][c], s[nt][c + 2]) > m[nt][c] + SLACK;
            if (__any_sync(FULL_MASK, grew)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float scale_o[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(s[nt][c], s[nt][c + 2]);
                        mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 16));
                        const float mn = fmaxf(m[nt][c], mx);
                        scale_o[c] = exp2_fast(m[nt][c] - finite_or_zero(mn));
                        m[nt][c] = mn;
                        l[nt][c] *= scale_o[c];
                    }
#pragma unroll
                    for (int kk = 0; kk < NK; ++kk)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[kk][nt][j] *= scale_o[j & 1];
                }
            }
            // p as hi + lo operands of the second product
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float mu = finite_or_zero(m[nt][c]) - P_SHIFT;
                    s[nt][c] = exp2_fast(s[nt][c] - mu);
                    s[nt][c + 2] = exp2_fast(s[nt][c + 2] - mu);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t hi = pack2<BF>(s[nt][2 * r], s[nt][2 * r + 1]);
                    const float2 back = unpack2<BF>(hi);
                    const uint32_t lo = pack2<BF>(s[nt][2 * r] - back.x, s[nt][2 * r + 1] - back.y);
                    ph[nt][r] = transpose_8x8(hi);
                    pl[nt][r] = transpose_8x8(lo);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                l[nt][0] += s[nt][0] + s[nt][2];
                l[nt][1] += s[nt][1] + s[nt][3];
            }

            if (KV != KV_E4M3) {
                const int key = (lane & 7) + ((lane >> 4) << 3);
                const uint32_t base = smem_addr(sv + key * ROW);
#pragma unroll
                for (int kk = 0; kk < NK; ++kk)
                    if (kk < nk) {
                        uint32_t v4[4];
                        ldsm_x4_t(v4, base + (((kk * 2 + ((lane >> 3) & 1)) ^ (key & 7)) << 4));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816<BF>(o[kk][nt], v4, ph[nt][0], ph[nt][1]);
                            mma16816<BF>(o[kk][nt], v4, pl[nt][0], pl[nt][1]);
                        }
                    }
            } else {
                // 32 dims at a time: the thread's four codes (dims 32j + 4g ..) of
                // keys 2t, 2t+1, 2t+8, 2t+9, interleaved into key pairs
#pragma unroll
                for (int j = 0; j < (DP + 31) / 32; ++j) {
                    uint32_t w[4];
                    const int col = j * 2 + (g >> 2);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int key = 2 * t + (r & 1) + (r >> 1) * 8;
                        const int sw = CHP >= 8 ? col ^ (((key >> 1) & 3) << 1) : col ^ (((key >> 1) & 1) << 1);
                        w[r] = *reinterpret_cast<const uint32_t*>(sv + key * ROW + sw * 16 + (g & 3) * 4);
                    }
                    uint32_t f[8];  // dims 4g + i: f[i] keys 2t, 2t+1; f[4 + i] keys 2t+8, 2t+9
                    e4m3x4_to_f16(__byte_perm(w[0], w[1], 0x5140), f[0], f[1]);
                    e4m3x4_to_f16(__byte_perm(w[0], w[1], 0x7362), f[2], f[3]);
                    e4m3x4_to_f16(__byte_perm(w[2], w[3], 0x5140), f[4], f[5]);
                    e4m3x4_to_f16(__byte_perm(w[2], w[3], 0x7362), f[6], f[7]);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t v4[4] = {f[2 * r], f[2 * r + 1], f[4 + 2 * r], f[4 + 2 * r + 1]};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816<false>(o[2 * j + r][nt], v4, ph[nt][0], ph[nt][1]);
                            mma16816<false>(o[2 * j + r][nt], v4, pl[nt][0], pl[nt][1]);
                        }
                    }
                }
            }
        }
        cp_async_wait<0>();

        // combine the warps: o to shared memory (each warp over its own ring),
        // weighted by exp2(m_warp - m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v = l[nt][c];
                v += __shfl_xor_sync(FULL_MASK, v, 4);
                v += __shfl_xor_sync(FULL_MASK, v, 8);
                v += __shfl_xor_sync(FULL_MASK, v, 16);
                if (g == 0) {
                    sm_m[warp * NH + nt * 8 + 2 * t + c] = m[nt][c];
                    sm_l[warp * NH + nt * 8 + 2 * t + c] = v;
                }
            }
        __syncwarp();
        float* so = reinterpret_cast<float*>(ring);  // [NH][SO]
#pragma unroll
        for (int kk = 0; kk < NK; ++kk)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int h = nt * 8 + 2 * t + (j & 1);
                    const int dim = KV == KV_E4M3 ? (kk >> 1) * 32 + 4 * g + (kk & 1) * 2 + (j >> 1)
                                                  : kk * 16 + g + (j >> 1) * 8;
                    so[h * SO + dim] = o[kk][nt][j];
                }
        __syncthreads();

        // factors of the warps' sums, once per head: exp2(m_warp - m)
        if (tid < NH) {
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < ATT_WARPS; ++w) mm = fmaxf(mm, sm_m[w * NH + tid]);
            const float mu = finite_or_zero(mm);
            float ll = 0.f;
#pragma unroll
            for (int w = 0; w < ATT_WARPS; ++w) {
                const float f = exp2_fast(sm_m[w * NH + tid] - mu);
                ll += f * sm_l[w * NH + tid];
                sm_m[w * NH + tid] = f;
            }
            head_ml[tid] = make_float2(mm, ll);
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == units;
        const int slot = 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0);
        const int vecs = heads * (a.D / 4);  // four dims a thread
        for (int e = tid; e < vecs; e += ATT_THREADS) {
            const int h = e / (a.D / 4), dim = (e - h * (a.D / 4)) * 4;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < ATT_WARPS; ++w)
                add_scaled(sum, sm_m[w * NH + h],
                           *reinterpret_cast<const float4*>(smem + (size_t)w * NST * 2 * HALF + (h * SO + dim) * 4));
            if (whole)
                store_head4<QBF>(a, b, head0 + h, dim, sum, head_ml[h], P_SHIFT);
            else
                *reinterpret_cast<float4*>(a.ws_o + ((int64_t)slot * a.hpi + h) * a.D + dim) = sum;
        }
        if (!whole) {
            if (tid < heads) reinterpret_cast<float2*>(a.ws_ml)[(int64_t)slot * a.hpi + tid] = head_ml[tid];
            // the pieces of this item belong to blocks c1 .. c2, the last ones
            // whose costs start before its first key and before its end
            const int c1 = (int)(((first_u + ATT_BEGIN + 1) * blocks - 1) / total);
            const int c2 = (int)(((first_u + cost) * blocks - 1) / total);
            join_pieces<QBF>(a, c1, c2, b, head0, heads, P_SHIFT, head_ml, reinterpret_cast<int*>(sm_warp));
        }
        __syncthreads();  // the ring and the flags are free again
        u = first_u + ATT_BEGIN + t1;
    }
}

// Blocks that a launch may have (pieces in the workspace): 160 SMs' worth.
static int attn_max_blocks(int D, int hpi) {
    const int nt = hpi > 8 ? 2 : 1;
    return 160 * att_blocks(D <= 64 ? 64 : D <= 128 ? 128 : 256, nt);
}

template <int DP, int NT, int KV, bool QBF>
static cudaError_t launch_attn(const AttnArgs& a, const DeviceInfo& di, cudaStream_t st) {
    constexpr int ES = KV == KV_E4M3 ? 1 : 2;
    const size_t smem = (size_t)ATT_WARPS * att_stages(DP, ES, NT) * 2 * ATT_STEP * DP * ES +
                        ATT_WARPS * att_stages(DP, ES, NT) * 4 + 2 * ATT_WARPS * NT * 8 * 4 + NT * 8 * 8 + 64 + (size_t)a.B * 8;
    auto kernel = paged_attention_kernel<DP, NT, KV, QBF>;
    static SmemOnce once;
    cudaError_t e = once.set(reinterpret_cast<const void*>(kernel), di.max_smem_optin);
    if (e != cudaSuccess) return e;
    if (smem > (size_t)di.max_smem_optin) return cudaErrorInvalidValue;
    int per_sm = (int)((size_t)di.smem_per_sm / (smem + 1024));
    per_sm = per_sm < 1 ? 1 : min(per_sm, att_blocks(DP, NT));
    const int grid = min(di.sm_count * per_sm, attn_max_blocks(a.D, a.hpi));
    return launch_after(kernel, dim3(grid), ATT_THREADS, smem, st, a);
}

template <int KV, bool QBF>
static cudaError_t launch_attn_kv(const AttnArgs& a, const DeviceInfo& di, cudaStream_t st) {
    const bool two = a.hpi > 8;
    if (a.D <= 64) return two ? launch_attn<64, 2, KV, QBF>(a, di, st) : launch_attn<64, 1, KV, QBF>(a, di, st);
    if (a.D <= 128) return two ? launch_attn<128, 2, KV, QBF>(a, di, st) : launch_attn<128, 1, KV, QBF>(a, di, st);
    return two ? launch_attn<256, 2, KV, QBF>(a, di, st) : launch_attn<256, 1, KV, QBF>(a, di, st);
}

// Query heads of one item: the group of a key-value head in equal parts of at
// most 16 (two N tiles; a third would not leave registers for D = 256).
int attn_heads_per_item(int G) {
    const int chunks = (G + 15) / 16;
    return (G + chunks - 1) / chunks;
}

size_t attn_workspace_bytes(int Hq, int Hkv, int D) {
    const size_t hpi = attn_heads_per_item(Hq / Hkv);
    return ATTN_COUNTER_BYTES + (size_t)2 * attn_max_blocks(D, (int)hpi) * hpi * (D + 2) * 4;
}

cudaError_t launch_paged_attention(AttnArgs a, int dtype, int cache_dtype, void* ws, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    a.err = di.err_word;
    a.G = a.Hq / a.Hkv;
    a.hpi = attn_heads_per_item(a.G);
    a.chunks = (a.G + a.hpi - 1) / a.hpi;
    int log2_page = 0;  // tok / page as a product: exact for tok < 2^31
    while ((int64_t(1) << log2_page) < a.page) ++log2_page;
    a.page_shift = 31 + log2_page;
    a.page_mul = (uint32_t)((uint64_t(1) << a.page_shift) / a.page + 1);
    a.out_aligned = reinterpret_cast<uintptr_t>(a.out) % 8 == 0;
    a.counters = static_cast<int*>(ws);
    a.ws_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + ATTN_COUNTER_BYTES);
    a.ws_o = a.ws_ml + (size_t)2 * attn_max_blocks(a.D, a.hpi) * a.hpi * 2;
    if (cache_dtype == MOE_E4M3)
        return dtype == MOE_BF16 ? launch_attn_kv<KV_E4M3, true>(a, di, st) : launch_attn_kv<KV_E4M3, false>(a, di, st);
    return dtype == MOE_BF16 ? launch_attn_kv<KV_BF16, true>(a, di, st) : launch_attn_kv<KV_F16, false>(a, di, st);
}

}  // namespace moedec
