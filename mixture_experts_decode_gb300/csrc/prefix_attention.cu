// prefix_attention.cu -- the part of a batch's attention that all its
// sequences share: every query row of every sequence against the keys and
// values of one long prefix, each read once for all of them, and the join with
// what each sequence has read of its own keys (attention.cu, `PART`).
//
// Mathematics.  For a key-value head the rows are the query heads of all
// sequences that read it, R = B * Hq / Hkv of them, 128 to a tile:
//   S [128 x KT] = Q [128 x D] K^T,   O [128 x D] += P [128 x KT] V
// with P = exp2(S * scale - m) and a running reference m and sum l per row,
// O and l rescaled only when some score passes m by SLACK.  The prefix is cut
// over the blocks; every block leaves (m, l, O) of its keys, and the join adds
// pieces by weights exp2(m_piece - m), in order, so the result does not depend
// on timing.
//
// Both products run on the tensor cores (tcgen05, accumulators in tensor
// memory): a row of S belongs to one thread, which reads it from tensor
// memory, needs no exchange for its maximum and sum, and writes P over it as
// the second product's A operand.  Two streams of jobs, a softmax warpgroup
// each, alternate on the tensor pipe: two row tiles on the same keys where
// there are more than 128 rows, else even and odd key tiles of one row tile.
//
// Rounding choices: scores, softmax and sums are FP32.  P is given to the
// second product as hi + lo, two 16-bit values, as in attention.cu: one
// rounding would cost as much as the output's own.  Where the output is BF16
// and the operands are FP16 (an E4M3 cache) hi alone is within 2^-11, an eighth
// of the output's rounding, and lo is left out.  A BF16 query against E4M3 keys
// goes to FP16 by a power of two per row, as there.
//
// Bound: HBM for few rows (the prefix once), the tensor pipe and the softmax
// for many.
#include <algorithm>

#include "block_common.cuh"
#include "decode_common.cuh"
#include "internal.h"

namespace moedec {

namespace {

constexpr int KV_BF16 = 0, KV_F16 = 1, KV_E4M3 = 2;
constexpr int PX_ROWS = 128;            // query rows of a tile (the MMA's M, a warpgroup's threads)
constexpr int PX_SOFT = 8;              // softmax warps (two warpgroups)
constexpr int PX_MMA = PX_SOFT;         // the warp that issues the products
constexpr int PX_KW = PX_SOFT + 1;      // first of four warps that bring K
constexpr int PX_VW = PX_KW + 4;        // first of four warps that bring V
constexpr int PX_THREADS = (PX_VW + 4) * 32;

// DB: blocks of 64 dims that hold a head.
constexpr int px_streams(int db) { return db == 4 ? 1 : 2; }  // (two sums of 256 columns would leave no room for scores)
constexpr int px_keys(int db) { return db == 4 ? 64 : 128; }  // keys of a tile
constexpr int px_stages(int db) { return db == 1 ? 4 : 2; }
constexpr int px_half(int db) { return db * px_keys(db) * 128; }  // bytes of a K (or V) tile

// Masks of live keys that are kept: the warps that write tile t's have waited
// for S(t - 2 - ST) or later, which was issued after the softmax of job
// t - 2 - 2 ST at the latest.
constexpr int px_masks(int db) { return 2 * px_stages(db) + 4; }

struct PxLayout {
    uint32_t k, v, koff, voff, live, back, bars, slot, abort, total;
};
constexpr PxLayout px_layout(int db) {
    PxLayout L{};
    uint32_t off = (uint32_t)px_streams(db) * db * PX_ROWS * 128;  // Q first
    L.k = off;     off += px_stages(db) * px_half(db);
    L.v = off;     off += px_stages(db) * px_half(db);
    L.koff = off;  off += 2 * 128 * 8;
    L.voff = off;  off += 2 * 128 * 8;
    L.live = off;  off += px_masks(db) * 16;
    L.back = off;  off += 2 * PX_ROWS * 4;
    L.bars = off;  off += (4 * px_stages(db) + 7) * 8;
    L.slot = off;  off += 8;
    L.abort = off; off += 8;
    L.total = off;
    return L;
}

__device__ __forceinline__ uint32_t swz(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)); }

// Matrix descriptor of a tile in the 128-byte swizzle: rows of 128 bytes, 8
// rows to a group of 1024 bytes (the stride offset).  K-major operands (Q, K:
// dims contiguous) ignore the leading offset; of an MN-major one (V: dims are
// the product's N) it is the distance between blocks of 64 dims.
__device__ __forceinline__ uint64_t px_desc(uint32_t saddr, uint32_t lead_bytes) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(lead_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// kind::f16: FP32 sums (bit 4), types of A and B (bits 7, 10: 1 for BF16), B
// MN-major (bit 16), N / 8, M / 16.
__device__ __forceinline__ uint32_t px_idesc(bool bf, bool b_mn, int n) {
    return (1u << 4) | (bf ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(PX_ROWS >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 (16) consecutive columns of the warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tm_ld32(uint32_t at, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
    wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tm_ld16(uint32_t at, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
    wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tm_st32(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
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
__device__ __forceinline__ bool mbar_done(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}
template <int ID>
__device__ __forceinline__ void four_warps_sync() {
    asm volatile("bar.sync %0, 128;" ::"n"(ID) : "memory");
}

}  // namespace

// A block: one key-value head, one group of row tiles, one run of key tiles.
// Roles: softmax warps 0 .. 7 (they also bring Q), the MMA warp, four warps
// that bring K tiles and four that bring V tiles (rows of pages by 16-byte
// asynchronous copies into the swizzle; E4M3 codes through registers, widened).
// Job j: scores and products of one row tile with one key tile, on score
// buffer j & 1; the MMA warp issues S(0) S(1) PV(0) S(2) PV(1) S(3) ...: the
// products of one thread run in order, so S(j + 2) may take the buffer that
// PV(j) reads.  Barriers: k_full / v_full (the bringing warps), k_empty /
// v_empty (commits), s_full (commit, and an arrival of the MMA thread that
// carries what it saw of the tile's live keys), p_full (softmax warps), o_done
// (commit of the stream's last PV).  Every wait is bounded; one that gives up
// raises `abort`, and every role goes to the end.
template <int DB, int KV, bool QBF>
__global__ void __launch_bounds__(PX_THREADS, 1) prefix_attention_kernel(const __grid_constant__ PrefixArgs a) {
    constexpr int NS = px_streams(DB), KT = px_keys(DB), ST = px_stages(DB), HALF = px_half(DB);
    constexpr bool BF = KV == KV_BF16;          // operand type of the products
    constexpr bool LO = !(KV == KV_E4M3 && QBF);  // P as hi + lo
    constexpr float P_SHIFT = BF ? 0.f : 14.f;
    constexpr float SLACK = BF ? 8.f : 1.f;  // FP16 holds 2^15 p
    constexpr PxLayout L = px_layout(DB);

    extern __shared__ __align__(1024) uint8_t px_smem[];
    uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(px_smem) + 1023) & ~uintptr_t(1023));
    uint64_t* const k_full = reinterpret_cast<uint64_t*>(sm + L.bars);
    uint64_t* const k_empty = k_full + ST;
    uint64_t* const v_full = k_full + 2 * ST;
    uint64_t* const v_empty = k_full + 3 * ST;
    uint64_t* const s_full = k_full + 4 * ST;
    uint64_t* const p_full = s_full + 2;
    uint64_t* const o_done = s_full + 4;
    uint64_t* const drained = s_full + 6;
    uint32_t* const live = reinterpret_cast<uint32_t*>(sm + L.live);  // [px_masks][4]
    float* const back = reinterpret_cast<float*>(sm + L.back);        // [rows]
    volatile int* const abort = reinterpret_cast<volatile int*>(sm + L.abort);

    const int tid = threadIdx.x, lane = tid & 31, warp = warp_index();
    // grid: splits fastest, so that blocks that read the same keys for
    // different rows run at the same time
    const int split = (int)blockIdx.x % a.splits;
    const int unit = (int)blockIdx.x / a.splits;
    const int kvh = unit % a.Hkv, group = unit / a.Hkv;
    const int R = a.B * a.G;
    const int row0 = group * NS * PX_ROWS;
    const int MT = NS == 2 && R - row0 > PX_ROWS ? 2 : 1;  // row tiles
    const int n_tiles = (a.len + KT - 1) / KT;
    const int tile0 = (int)((int64_t)n_tiles * split / a.splits);
    const int tiles = (int)((int64_t)n_tiles * (split + 1) / a.splits) - tile0;
    const int jobs = tiles * MT;
    const int D = a.D;

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 2);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
        }
        mbar_init(drained, 1);
        *abort = 0;
        mbar_init_fence();
    }
    if (warp == PX_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_addr(sm + L.slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    after_previous();

    // Q, by the softmax warps: CH lanes of 16 bytes a row
    if (warp < PX_SOFT) {
        const int CH = D / 8;
        const bool flip = a.scale_log2 < 0.f;  // the products take |scale|, q its sign
        const int per = CH <= 8 ? 8 : CH <= 16 ? 16 : 32;  // lanes of a row
        const int c = lane & (per - 1);
        const int rows = NS * PX_ROWS;
#pragma unroll 4
        for (int r = tid / per; r < rows; r += PX_SOFT * 32 / per) {
            const int row = row0 + r;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (row < R && c < CH) {
                const int b = row / a.G, h = kvh * a.G + (row - b * a.G);
                v = ld_128(static_cast<const uint16_t*>(a.q) + (int64_t)b * a.q_sb + (int64_t)h * a.q_sh + c * 8);
            }
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (KV == KV_E4M3 && QBF) {
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p = bf16x2_to_float2(w[i]);
                    amax = fmaxf(amax, fmaxf(fabsf(p.x), fabsf(p.y)));
                }
                for (int o = per / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, o));
                // 2^e <= amax < 2^(e+1); q * 2^(9-e), undone in the scale
                int e = (int)(__float_as_uint(amax) >> 23) - 127;
                e = max(-100, min(e, 127));
                const float fwd = __uint_as_float((uint32_t)(127 + min(9 - e, 109)) << 23);
                if (c == 0) back[r] = __uint_as_float((uint32_t)(127 - min(9 - e, 109)) << 23);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p = bf16x2_to_float2(w[i]);
                    w[i] = pack2<false>(p.x * fwd, p.y * fwd);
                }
            }
            if (c < CH) {
                const uint32_t s = flip ? 0x80008000u : 0u;
                *reinterpret_cast<uint4*>(sm + ((r >> 7) * DB + (c >> 3)) * (PX_ROWS * 128) + swz(r & 127, c & 7)) =
                    make_uint4(w[0] ^ s, w[1] ^ s, w[2] ^ s, w[3] ^ s);
            }
        }
        fence_proxy_async();
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + L.slot);

    if (warp == PX_MMA) {
        if (lane == 0) {
            const uint32_t q0 = smem_addr(sm), k0 = smem_addr(sm + L.k), v0 = smem_addr(sm + L.v);
            const uint32_t id_s = px_idesc(BF, false, KT), id_o = px_idesc(BF, true, D);
            bool ok = true;
            auto scores = [&](int j) {
                const int t = MT == 2 ? j >> 1 : j, st = t % ST;
                if (!mbar_wait_abort(&k_full[st], (t / ST) & 1, abort)) return false;
                fence_after();
                const uint32_t q = q0 + (MT == 2 ? (j & 1) * DB * (PX_ROWS * 128) : 0);
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + (j & 1) * 128, px_desc(q + (kk >> 2) * (PX_ROWS * 128) + (kk & 3) * 32, 16),
                           px_desc(k0 + st * HALF + (kk >> 2) * (KT * 128) + (kk & 3) * 32, 16), id_s, kk > 0);
                mma_commit(&s_full[j & 1]);
                mbar_arrive(&s_full[j & 1]);
                if (MT == 1 || (j & 1)) mma_commit(&k_empty[st]);
                return true;
            };
            for (int j = 0; j < 2 && j < jobs && ok; ++j) ok = scores(j);
            for (int j = 0; j < jobs && ok; ++j) {
                const int t = MT == 2 ? j >> 1 : j, st = t % ST, s = NS == 2 ? j & 1 : 0;
                if (!mbar_wait_abort(&p_full[j & 1], (j >> 1) & 1, abort) ||
                    !mbar_wait_abort(&v_full[st], (t / ST) & 1, abort)) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t o = tmem + 256 + s * 128, p = tmem + (j & 1) * 128;
                const bool first = j < NS;
                for (int kk = 0; kk < KT / 16; ++kk) {
                    const uint64_t v = px_desc(v0 + st * HALF + kk * 2048, KT * 128);
                    const uint32_t pa = p + (kk >> 1) * 32 + (kk & 1) * 8;
                    mma_ts(o, pa, v, id_o, !first || kk > 0);
                    if (LO) mma_ts(o, pa + 16, v, id_o, 1u);
                }
                mma_commit(&o_done[s]);
                if (MT == 1 || (j & 1)) mma_commit(&v_empty[st]);
                if (j + 2 < jobs) ok = scores(j + 2);
            }
            // products already issued finish before tensor memory is freed
            mma_commit(drained);
            mbar_wait(drained, 0);
        }
        __syncwarp();
    } else if (warp < PX_SOFT) {
        const int s = NS == 2 ? warp >> 2 : 0;
        const int r = (NS == 2 && MT == 2 ? s * PX_ROWS : 0) + (warp & 3) * 32 + lane;  // row of the group
        if (NS == 2 || warp < 4) {
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t o_at = tmem + lanes + 256 + s * 128;
            float sl = fabsf(a.scale_log2);
            if (KV == KV_E4M3 && QBF) sl *= back[r];
            sl = fmaxf(sl, 0x1p-126f);  // (masked scores of -inf stay so with a scale of 0)
            float m = -INFINITY, l = 0.f;
            int c = 0;  // jobs of this stream so far
            bool ok = true;
            for (int j = s; j < jobs; j += NS, ++c) {
                const int t = MT == 2 ? j >> 1 : j;
                if (!__all_sync(FULL_MASK, mbar_wait_abort(&s_full[j & 1], (j >> 1) & 1, abort))) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t s_at = tmem + lanes + (j & 1) * 128;
                const uint32_t* mask = live + (t % px_masks(DB)) * 4;
                bool all = true;
#pragma unroll
                for (int i = 0; i < KT / 32; ++i) all &= mask[i] == FULL_MASK;
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < KT / 32; ++i) {
                    float v[32];
                    tm_ld32(s_at + i * 32, v);
                    if (!all) {
                        const uint32_t on = mask[i];
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = on >> e & 1u ? v[e] : -INFINITY;
                    }
                    float m0 = v[0], m1 = v[1];
#pragma unroll
                    for (int e = 2; e < 32; e += 2) m0 = fmaxf(m0, v[e]), m1 = fmaxf(m1, v[e + 1]);
                    mx = fmaxf(mx, fmaxf(m0, m1));
                }
                mx *= sl;
                if (__any_sync(FULL_MASK, mx > m + SLACK)) {
                    const float mn = fmaxf(m, mx);
                    const float f = exp2_fast(m - finite_or_zero(mn));
                    m = mn;
                    l *= f;
                    if (c > 0) {
                        if (!__all_sync(FULL_MASK, mbar_wait_abort(&o_done[s], (c - 1) & 1, abort))) {
                            ok = false;
                            break;
                        }
                        fence_after();
                        for (int d = 0; d < D; d += 16) {
                            float o[16];
                            uint32_t w[16];
                            tm_ld16(o_at + d, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);
                            tm_st16(o_at + d, w);
                        }
                        wait_st();
                    }
                }
                const float mu = finite_or_zero(m) - P_SHIFT;
                float l0 = 0.f, l1 = 0.f;
#pragma unroll
                for (int i = 0; i < KT / 32; ++i) {
                    float v[32];
                    tm_ld32(s_at + i * 32, v);
                    if (!all) {
                        const uint32_t on = mask[i];
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = on >> e & 1u ? v[e] : -INFINITY;
                    }
                    uint32_t w[32];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float p0 = exp2_fast(fmaf(v[2 * e], sl, -mu)), p1 = exp2_fast(fmaf(v[2 * e + 1], sl, -mu));
                        l0 += p0, l1 += p1;
                        w[e] = pack2<BF>(p0, p1);
                        if (LO) {
                            const float2 h = unpack2<BF>(w[e]);
                            w[16 + e] = pack2<BF>(p0 - h.x, p1 - h.y);
                        }
                    }
                    if (LO) {
                        tm_st32(s_at + i * 32, w);
                    } else {
                        uint32_t hi[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) hi[e] = w[e];
                        tm_st16(s_at + i * 32, hi);
                    }
                }
                l += l0 + l1;
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[j & 1]);
            }
            // the piece: (m, l) and O of this row, O only where some job ran
            if (ok && c > 0) ok = __all_sync(FULL_MASK, mbar_wait_abort(&o_done[s], (c - 1) & 1, abort));
            const int row = row0 + r;
            const int piece = MT == 1 && NS == 2 ? 2 * split + s : split;
            const int64_t at = ((int64_t)kvh * a.pieces + piece) * R + row;
            if (row < R)
                reinterpret_cast<float2*>(a.ws_ml)[at] = ok && c > 0 ? make_float2(m - P_SHIFT, l) : make_float2(-INFINITY, 0.f);
            if (ok && c > 0) {
                fence_after();
                float* out = a.ws_o + at * D;
                for (int d = 0; d < D; d += 16) {
                    float o[16];
                    tm_ld16(o_at + d, o);
                    if (row < R) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4*>(out + d + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
            }
        }
    } else {
        // ---------------- K and V tiles, four warps each ----------------
        const bool is_v = warp >= PX_VW;
        const int pt = tid - (is_v ? PX_VW : PX_KW) * 32;  // 0 .. 127
        uint64_t* const full = is_v ? v_full : k_full;
        uint64_t* const empty = is_v ? v_empty : k_empty;
        int64_t* const offs = reinterpret_cast<int64_t*>(sm + (is_v ? L.voff : L.koff));
        uint8_t* const ring = sm + (is_v ? L.v : L.k);
        constexpr int ES = KV == KV_E4M3 ? 1 : 2;
        const int64_t sp = (is_v ? a.v_sp : a.k_sp) * ES, stt = (is_v ? a.v_st : a.k_st) * ES;
        const uint8_t* const src = static_cast<const uint8_t*>(is_v ? a.v : a.k) + (int64_t)kvh * (is_v ? a.v_sh : a.k_sh) * ES;

        // Thread i finds key i's row, a tile ahead of its use.
        int pg = 0, off = 0;
        auto find = [&](int t) {
            if (t >= tiles || pt >= KT) return;
            const int key = min((tile0 + t) * KT + pt, a.len - 1);
            const int pi = (int)(((uint64_t)(uint32_t)key * a.page_mul) >> a.page_shift);
            off = key - pi * a.page;
            pg = a.table[pi];
        };
        // Offsets of tile t's rows (-1: not live) to all four warps.
        auto publish = [&](int t) {
            if (pt < KT) {
                const bool known = pg >= 0 && pg < a.num_pages;
                if (!known) atomicOr(a.err, MOE_DEVERR_PAGE);
                const bool have = known && (tile0 + t) * KT + pt < a.len;
                offs[(t & 1) * 128 + pt] = have ? pg * sp + off * stt : -1;
                const uint32_t word = __ballot_sync(FULL_MASK, have);
                if (!is_v && lane == 0) live[(t % px_masks(DB)) * 4 + (pt >> 5)] = word;
            }
            if (is_v)
                four_warps_sync<2>();
            else
                four_warps_sync<1>();
        };
        auto arrive = [&](int t) {
            fence_proxy_async();  // this thread's part of the tile, before the tensor cores read it
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[t % ST]);
        };
        find(0);
        bool ok = true;
        if (KV != KV_E4M3) {
            const int CH = D / 8, per = 128 / CH;  // rows that the warps copy at once
            const int c = pt % CH, r0 = pt / CH;
            const uint32_t col = (c >> 3) * (KT * 128);
            int sent = 0;  // tiles whose copies have been announced
            for (int t = 0; t < tiles; ++t) {
                publish(t);
                find(t + 1);
                const int st = t % ST;
                if (t >= ST && ok) {
                    const uint32_t par = ((t / ST) - 1) & 1;
                    // nothing to issue yet: what is on its way is announced first
                    if (!__all_sync(FULL_MASK, mbar_done(&empty[st], par))) {
                        cp_async_wait<0>();
                        for (; sent < t; ++sent) arrive(sent);
                        ok = __all_sync(FULL_MASK, mbar_wait_abort(&empty[st], par, abort));
                    }
                }
                if (!ok) continue;  // (the four warps stay together at publish)
                uint8_t* const dst = ring + st * HALF + col;
                const int64_t* const o = offs + (t & 1) * 128;
                if (r0 < per)
#pragma unroll 4
                    for (int row = r0; row < KT; row += per) {
                        const int64_t at = o[row];
                        cp_async_16_zfill(dst + swz(row, c & 7), src + (at < 0 ? 0 : at) + c * 16, at < 0 ? 0 : 16);
                    }
                cp_async_commit();
                if (sent < t) {  // (at most tile t - 1 is left)
                    cp_async_wait<1>();
                    for (; sent < t; ++sent) arrive(sent);
                }
            }
            cp_async_wait<0>();
            if (ok)
                for (; sent < tiles; ++sent) arrive(sent);
        } else {
            // 16 codes a thread at a time, the next tile's in registers
            constexpr int PER = KT * DB * 4 / 128;  // pieces of 16 codes a thread has of a tile at most
            const int CH = D / 16;
            uint4 next[PER];
            int rows[PER], cols[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                rows[i] = (pt + i * 128) / CH;
                cols[i] = pt + i * 128 - rows[i] * CH;
            }
            auto load = [&](int t) {
                const int64_t* const o = offs + (t & 1) * 128;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int row = rows[i], c = cols[i];
                    const int64_t at = row < KT ? o[row] : -1;
                    next[i] = at < 0 ? make_uint4(0u, 0u, 0u, 0u) : ld_128(src + at + c * 16);
                }
            };
            if (tiles > 0) {
                publish(0);
                find(1);
                load(0);
            }
            for (int t = 0; t < tiles; ++t) {
                const int st = t % ST;
                uint4 cur[PER];
#pragma unroll
                for (int i = 0; i < PER; ++i) cur[i] = next[i];
                if (t + 1 < tiles) {
                    publish(t + 1);
                    find(t + 2);
                    load(t + 1);
                }
                if (t >= ST && ok) ok = __all_sync(FULL_MASK, mbar_wait_abort(&empty[st], ((t / ST) - 1) & 1, abort));
                if (!ok) continue;  // (the four warps stay together at publish)
                uint8_t* const dst = ring + st * HALF;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int row = rows[i], c = cols[i];
                    if (row < KT) {
                        uint32_t w[8];
                        e4m3x4_to_f16(cur[i].x, w[0], w[1]);
                        e4m3x4_to_f16(cur[i].y, w[2], w[3]);
                        e4m3x4_to_f16(cur[i].z, w[4], w[5]);
                        e4m3x4_to_f16(cur[i].w, w[6], w[7]);
                        uint8_t* const d = dst + (c >> 2) * (KT * 128);
                        *reinterpret_cast<uint4*>(d + swz(row, (2 * c) & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(d + swz(row, (2 * c + 1) & 7)) = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
                arrive(t);
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == PX_MMA) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
    if (tid == 0 && *abort) atomicOr(a.err, MOE_DEVERR_TIMEOUT);
}

// Every output from its pieces: the prefix's, in the order of its runs, where
// the sequence shares it, then the sequence's own.  Four dims a thread, eight
// pieces' loads in flight; a piece of weight 0 may hold anything.
template <bool QBF>
__global__ void __launch_bounds__(128) prefix_join_kernel(const __grid_constant__ PrefixArgs a) {
    after_previous();
    const int vecs = a.D / 4;
    const int64_t e = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (e >= (int64_t)a.B * a.Hq * vecs) return;
    const int64_t bh = e / vecs;
    const int dim = (int)(e - bh * vecs) * 4;
    const int b = (int)(bh / a.Hq), h = (int)(bh - (int64_t)b * a.Hq);
    const int kvh = h / a.G, R = a.B * a.G, row = b * a.G + (h - kvh * a.G);
    int np = 0;
    if (min((int64_t)a.lens[b], a.cap) >= a.len && (!a.shares || a.shares[b])) {
        const int g0 = row / a.group_rows * a.group_rows;
        np = a.group_rows > PX_ROWS && R - g0 <= PX_ROWS ? 2 * a.splits : a.splits;
    }
    const float2* const mls = reinterpret_cast<const float2*>(a.ws_ml) + (int64_t)kvh * a.pieces * R + row;
    const float* const os = a.ws_o + ((int64_t)kvh * a.pieces * R + row) * a.D + dim;
    const float2 own_ml = reinterpret_cast<const float2*>(a.own_ml)[bh];
    const float4 own = *reinterpret_cast<const float4*>(a.own_o + bh * a.D + dim);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    auto scale = [&](float mn) {
        const float old = exp2_fast(m - finite_or_zero(mn));
        m = mn;
        l *= old;
        sum.x *= old, sum.y *= old, sum.z *= old, sum.w *= old;
    };
    auto add = [&](float2 ml, const float4& v) {
        const float f = exp2_fast(ml.x - finite_or_zero(m));
        if (f == 0.f) return;
        l += f * ml.y;
        sum.x += f * v.x, sum.y += f * v.y, sum.z += f * v.z, sum.w += f * v.w;
    };
#pragma unroll 1
    for (int p0 = 0; p0 < np; p0 += 8) {
        float4 v[8];
        float2 ml[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t at = (int64_t)min(p0 + i, np - 1) * R;
            ml[i] = mls[at];
            v[i] = *reinterpret_cast<const float4*>(os + at * a.D);
        }
        float mn = m;
#pragma unroll
        for (int i = 0; i < 8; ++i) mn = fmaxf(mn, ml[i].x);
        scale(mn);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (p0 + i < np) add(ml[i], v[i]);
    }
    scale(fmaxf(m, own_ml.x));
    add(own_ml, own);
    const float f = l == 0.f ? 0.f : a.v_scale / l;
    const uint32_t lo = pack2<QBF>(sum.x * f, sum.y * f), hi = pack2<QBF>(sum.z * f, sum.w * f);
    uint16_t* const out = static_cast<uint16_t*>(a.out) + bh * a.D + dim;
    if (a.out_aligned) {
        *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
    } else {
        out[0] = (uint16_t)lo, out[1] = (uint16_t)(lo >> 16);
        out[2] = (uint16_t)hi, out[3] = (uint16_t)(hi >> 16);
    }
    if (dim == 0 && a.lse) a.lse[bh] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

static int px_db(int D) { return D <= 64 ? 1 : D <= 128 ? 2 : 4; }
static int px_group_rows(int D) { return px_streams(px_db(D)) * PX_ROWS; }

// Runs that the prefix is cut into: the number that ends first, when a block's
// time is its key tiles and about four of them for beginning and end, and
// blocks beyond the SMs' number take another round.
static int px_splits(int units, int tiles, int sms) {
    int best = 1;
    double least = 1e300;
    for (int s = 1; s <= tiles && (s == 1 || (int64_t)units * s <= PX_MAX_BLOCKS); ++s) {
        const double rounds = (double)(((int64_t)units * s + sms - 1) / sms);
        const double cost = rounds * ((tiles + s - 1) / s + 4) + 0.05 * s;
        if (cost < least) least = cost, best = s;
    }
    return best;
}

static int px_units(int B, int G, int Hkv, int D) { return Hkv * ((B * G + px_group_rows(D) - 1) / px_group_rows(D)); }

// The pieces (behind the own part's workspace): own (m, l) and O, and the
// prefix's for the largest number of runs, of this batch or a smaller one (a
// smaller one may be cut into more runs).
size_t prefix_workspace_bytes(int B, int Hq, int Hkv, int D) {
    const int G = Hq / Hkv, R = B * G, group = px_group_rows(D);
    size_t most = 0;
    for (int g = 1; (g - 1) * group < R; ++g) {
        const size_t rows = (size_t)Hkv * std::min(R, g * group);
        most = std::max(most, rows * 2 * std::max(1, PX_MAX_BLOCKS / (Hkv * g)));
    }
    return ((size_t)B * Hq + most) * (D + 2) * 4;
}

template <int DB, int KV, bool QBF>
static cudaError_t launch_px(const PrefixArgs& a, const DeviceInfo& di, int grid, cudaStream_t st) {
    constexpr size_t smem = px_layout(DB).total + 1024;
    static_assert(smem <= 227 * 1024, "a block's shared memory");
    auto kernel = prefix_attention_kernel<DB, KV, QBF>;
    static SmemOnce once;
    const cudaError_t e = once.set(reinterpret_cast<const void*>(kernel), di.max_smem_optin);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(grid), PX_THREADS, smem, st, a);
}

template <int KV, bool QBF>
static cudaError_t launch_px_kv(const PrefixArgs& a, const DeviceInfo& di, int grid, cudaStream_t st) {
    switch (px_db(a.D)) {
        case 1: return launch_px<1, KV, QBF>(a, di, grid, st);
        case 2: return launch_px<2, KV, QBF>(a, di, grid, st);
        default: return launch_px<4, KV, QBF>(a, di, grid, st);
    }
}

cudaError_t launch_shared_prefix(PrefixArgs a, const AttnArgs& own, int dtype, int cache_dtype, void* ws, cudaStream_t st) {
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    a.err = di.err_word;
    a.G = a.Hq / a.Hkv;
    a.group_rows = px_group_rows(a.D);
    a.out_aligned = reinterpret_cast<uintptr_t>(a.out) % 8 == 0;
    int log2_page = 0;  // key / page as a product: exact for key < 2^31
    while ((int64_t(1) << log2_page) < a.page) ++log2_page;
    a.page_shift = 31 + log2_page;
    a.page_mul = (uint32_t)((uint64_t(1) << a.page_shift) / a.page + 1);
    const int units = px_units(a.B, a.G, a.Hkv, a.D), KT = px_keys(px_db(a.D));
    a.splits = px_splits(units, (a.len + KT - 1) / KT, di.sm_count);
    a.pieces = a.group_rows > PX_ROWS ? 2 * a.splits : a.splits;
    const size_t rows = (size_t)a.B * a.Hq;
    char* const base = static_cast<char*>(ws) + (attn_workspace_bytes(a.Hq, a.Hkv, a.D) + 255) / 256 * 256;
    a.own_o = reinterpret_cast<float*>(base);
    a.ws_o = a.own_o + rows * a.D;
    a.ws_ml = a.ws_o + rows * a.pieces * a.D;
    a.own_ml = a.ws_ml + rows * a.pieces * 2;

    AttnArgs o = own;
    o.first = a.len, o.shares = a.shares, o.part_o = a.own_o, o.part_ml = a.own_ml;
    e = launch_paged_attention(o, dtype, cache_dtype, ws, st);
    if (e != cudaSuccess) return e;
    const int grid = units * a.splits;
    if (cache_dtype == MOE_E4M3)
        e = dtype == MOE_BF16 ? launch_px_kv<KV_E4M3, true>(a, di, grid, st) : launch_px_kv<KV_E4M3, false>(a, di, grid, st);
    else
        e = dtype == MOE_BF16 ? launch_px_kv<KV_BF16, true>(a, di, grid, st) : launch_px_kv<KV_F16, false>(a, di, grid, st);
    if (e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)((rows * (a.D / 4) + 127) / 128);
    return dtype == MOE_BF16 ? launch_after(prefix_join_kernel<true>, dim3(blocks), 128, 0, st, a)
                             : launch_after(prefix_join_kernel<false>, dim3(blocks), 128, 0, st, a);
}

}  // namespace moedec
