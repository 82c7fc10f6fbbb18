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
// rounding would cost as much as the output's own, and shows where values
// cancel (a BF16 output over an E4M3 cache with hi alone, FP16, differed from
// the plain form's by a relative 9e-4 in place of 1e-4; 64 x 65536 tokens then
// took 161 us in place of 199).  FP16 operands hold 2^7 p, with room for a
// reference that is 2^8 too low, so that weights below 2^-31 of the largest of a
// block's run are lost; attention.cu keeps them to 2^-38, but there the
// reference moves at every 2 that it is passed by, which is a round trip
// through tensor memory here (64 x 65536: 235 us).  A BF16 query against E4M3
// keys goes to FP16 by a power of two per row, as there.
//
// Bound: HBM for few rows (the prefix once); for many the chain score product,
// softmax, value product, score product of a stream, with the tensor pipe active
// half of the time; with few key tiles a block, what is around that: own keys,
// pieces and join.  Measured, whole calls: 64 sequences over 65536 tokens, 64 / 8
// heads of 128, E4M3 199 us (691 TFLOP/s; one launch of the paged kernel 1000), 191
// with an FP16 query; 32 over 8192, 32 / 4 of 128, BF16, chats of up to 1500 tokens
// 29.6 us (45), heads of 192 and 256, 400 own tokens 36 and 39 us (124); 300 over
// 9600, 16 / 2 of 64, FP16 48.9 us (142), of which own keys 18 and the join 10.
#include <algorithm>
#include <type_traits>

#include "block_common.cuh"
#include "decode_common.cuh"
#include "internal.h"

namespace moedec {

namespace {

constexpr int PX_ROWS = 128;            // query rows of a tile (the MMA's M, a warpgroup's threads)
constexpr int PX_SOFT = 8;              // softmax warps (two warpgroups)
constexpr int PX_MMA = PX_SOFT;         // the warp that issues the products
constexpr int PX_KW = PX_SOFT + 1;      // first of two warps that bring K
constexpr int PX_VW = PX_KW + 2;        // first of two warps that bring V
constexpr int PX_BRING = 64;            // threads of each
constexpr int PX_THREADS = (PX_VW + 2) * 32;

// DB: blocks of 64 dims that hold a head.
constexpr int px_streams(int db) { return db == 4 ? 1 : 2; }  // (two sums of 256 columns would leave no room for scores)
constexpr int px_keys(int db) { return db == 4 ? 64 : 128; }  // keys of a tile
constexpr int px_half(int db) { return db * px_keys(db) * 128; }  // bytes of a K (or V) tile of 16-bit values
// Stages of 16-bit tiles, and for an E4M3 cache of codes in front of them.  A
// widened K tile is wanted again only when the softmax between two uses is over,
// so one stage does where room is short; V's next tile is wanted as soon as the
// last is let go, so it has two, and one of codes, which the whole time of a
// tile is there to fill (64 x 65536 tokens, when a weight was one 16-bit value:
// 166 us; with one of V and two of its codes 182).
constexpr int px_k_stages(int db, bool e4) { return db == 1 ? (e4 ? 2 : 4) : (e4 ? 1 : 2); }
constexpr int px_v_stages(int db, bool e4) { return db == 1 && !e4 ? 4 : 2; }
constexpr int px_k_codes(int db, bool e4) { return !e4 ? 0 : db == 1 ? 3 : 2; }
constexpr int px_v_codes(int db, bool e4) { return !e4 ? 0 : db == 1 ? 3 : 1; }
// Masks of live keys that are kept: when tile t's is written, the scores of the
// tile a stage count before it have been issued, so the softmax of the tile two
// before that is over.
constexpr int px_masks(int db, bool e4) { return px_k_stages(db, e4) + px_k_codes(db, e4) + 4; }

constexpr int PX_PAGES = 512;  // pages, of K and of V, whose places shared memory holds

struct PxLayout {
    uint32_t k, v, codes, pages, rows, live, back, bars, slot, abort, total;
};
constexpr PxLayout px_layout(int db, bool e4) {
    PxLayout L{};
    uint32_t off = (uint32_t)px_streams(db) * db * PX_ROWS * 128;  // Q first
    L.k = off;     off += px_k_stages(db, e4) * px_half(db);
    L.v = off;     off += px_v_stages(db, e4) * px_half(db);
    L.codes = off; off += (px_k_codes(db, e4) + px_v_codes(db, e4)) * (px_half(db) / 2);
    L.pages = off; off += 2 * PX_PAGES * 8;
    L.rows = off;  off += 2 * 2 * 128 * 8;
    L.live = off;  off += px_masks(db, e4) * 16;
    L.back = off;  off += 2 * PX_ROWS * 4;
    L.bars = off;  off += (2 * px_k_stages(db, e4) + 2 * px_v_stages(db, e4) + 14) * 8;
    L.slot = off;  off += 8;
    L.abort = off; off += 8;
    L.total = off;
    return L;
}

__device__ __forceinline__ uint32_t swz(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)); }

// Matrix descriptor of a tile in the 128-byte swizzle: rows of 128 bytes, 8
// rows to a group of 1024 bytes (the stride offset, in the constant upper
// half).  K-major operands (Q, K: dims contiguous) ignore the leading offset;
// of an MN-major one (V: dims are the product's N) it is the distance between
// blocks of 64 dims.  An address moves on by adding to the lower half.
constexpr uint32_t PX_DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t px_desc_lo(uint32_t saddr, uint32_t lead_bytes) {
    return ((saddr >> 4) & 0x3FFFu) | ((lead_bytes >> 4) << 16);
}
// kind::f16: FP32 sums (bit 4), types of A and B (bits 7, 10: 1 for BF16), B
// MN-major (bit 16), N / 8, M / 16.
__device__ __forceinline__ uint32_t px_idesc(bool bf, bool b_mn, int n) {
    return (1u << 4) | (bf ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(PX_ROWS >> 4) << 24);
}
// Products and commits: the whole warp comes here, so that addresses stay in
// uniform registers, and its leader (the same lane every time) issues.
__device__ __forceinline__ uint32_t leader_lane() {
    uint32_t e;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
    return e;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p, q; .reg .b64 a, b;\n\t"
        "setp.ne.b32 q, %0, 0; setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%2, %6}; mov.b64 b, {%3, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, p; }" ::"r"(lead), "r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc),
        "r"(acc), "n"(PX_DESC_HI)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p, q; .reg .b64 b;\n\t"
        "setp.ne.b32 q, %0, 0; setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%3, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %4, p; }" ::"r"(lead), "r"(d), "r"(a), "r"(b_lo), "r"(idesc),
        "r"(acc), "n"(PX_DESC_HI)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(smem_addr(bar)), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 (16) consecutive columns of the warp's 32 lanes of tensor memory.  A
// load's registers hold its values from the wait on.
__device__ __forceinline__ void tm_ld32(uint32_t at, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tm_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// p - h for the two 16-bit values h of a word, each in one instruction.
template <bool BF>
__device__ __forceinline__ float2 rest2(float2 p, uint32_t h) {
    float2 r;
    if (BF)
        asm("{ .reg .b16 a, b, o; mov.b32 {a, b}, %4; mov.b16 o, 0xbf80;\n\t"
            "fma.rn.f32.bf16 %0, a, o, %2; fma.rn.f32.bf16 %1, b, o, %3; }"
            : "=f"(r.x), "=f"(r.y)
            : "f"(p.x), "f"(p.y), "r"(h));
    else
        asm("{ .reg .b16 a, b, o; mov.b32 {a, b}, %4; mov.b16 o, 0xbc00;\n\t"
            "fma.rn.f32.f16 %0, a, o, %2; fma.rn.f32.f16 %1, b, o, %3; }"
            : "=f"(r.x), "=f"(r.y)
            : "f"(p.x), "f"(p.y), "r"(h));
    return r;
}
// With the lane `bit` away: a lane whose bit is clear gives b and gets the
// other's a in its place, the other one the reverse.
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b, bool upper, int bit) {
    const uint32_t got = __shfl_xor_sync(FULL_MASK, upper ? a : b, bit);
    if (upper)
        a = got;
    else
        b = got;
}
// The barrier gets an arrival of this thread when its copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// An ordinary load past L1 (the inputs may be newer than L1's lines where the
// kernel begins before its predecessor's end).
__device__ __forceinline__ uint4 ld_128_l2(const void* p) {
    uint4 r;
    asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}
}  // namespace

// A block: one key-value head, one group of row tiles, one run of key tiles.
// Roles: softmax warps 0 .. 7 (they also bring Q), the MMA warp, two warps that
// bring K tiles and two that bring V tiles (rows of pages by 16-byte
// asynchronous copies into the swizzle; E4M3 codes into a stage of their own,
// widened from there).
// Job j: scores and products of one row tile with one key tile, on score
// buffer j & 1.  The MMA warp issues S(0) S(1) PV(0) S(2) PV(1) S(3) ..., PV in
// two halves of the keys, each as soon as its weights are there, and S(j + 2)
// when PV(j), which reads its weights from the same buffer, is done (products
// of different shapes and accumulators are not promised to run in order; the
// wait costs some 10 % at 64 x 65536 tokens).
// Barriers: q_full, k_full / v_full (those that bring; their writes are generic,
// so the MMA warp fences before the tensor cores read), k_empty / v_empty
// (commits), s_full (commit, and an arrival of the MMA warp that carries what it
// saw of the tile's live keys), p_full (softmax warps, per half), h_done /
// o_done (commits of PV's halves), last (a commit behind a stream's last PV: at
// the end o_done may be one phase or two past the one a warp has seen, and a
// parity tells neither).  Every wait is bounded; one that gives up
// raises `abort`, and every role goes to the end.
// The kernel does not wait for its predecessor, the own keys' kernel, which
// lets it start after everything before that one has completed; it does so at
// its end, so that the join behind it finds both.
template <int DB, int KV, bool QBF>
__global__ void __launch_bounds__(PX_THREADS, 1) prefix_attention_kernel(const __grid_constant__ PrefixArgs a) {
    constexpr bool E4 = KV == KV_E4M3;
    constexpr int NS = px_streams(DB), KT = px_keys(DB), HALF = px_half(DB), MASKS = px_masks(DB, E4);
    constexpr int KS = px_k_stages(DB, E4), VS = px_v_stages(DB, E4);
    constexpr bool BF = KV == KV_BF16;          // operand type of the products
    constexpr float P_SHIFT = BF ? 0.f : 7.f;
    constexpr float SLACK = 8.f;  // (FP16 holds up to 2^15)
    constexpr PxLayout L = px_layout(DB, E4);

    extern __shared__ __align__(1024) uint8_t px_smem[];
    uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(px_smem) + 1023) & ~uintptr_t(1023));
    uint64_t* const k_full = reinterpret_cast<uint64_t*>(sm + L.bars);
    uint64_t* const k_empty = k_full + KS;
    uint64_t* const v_full = k_empty + KS;
    uint64_t* const v_empty = v_full + VS;
    uint64_t* const s_full = v_empty + VS;
    uint64_t* const p_full = s_full + 2;
    uint64_t* const o_done = s_full + 6;  // (p_full: [buffer][half])
    uint64_t* const h_done = s_full + 8;
    uint64_t* const q_full = s_full + 10;
    uint64_t* const drained = s_full + 11;
    uint64_t* const last = s_full + 12;  // [stream], of one phase
    uint32_t* const live = reinterpret_cast<uint32_t*>(sm + L.live);  // [MASKS][4]
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
        for (int i = 0; i < KS; ++i) {
            mbar_init(&k_full[i], E4 ? 2 : PX_BRING + 2);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < VS; ++i) {
            mbar_init(&v_full[i], E4 ? 2 : PX_BRING);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 2);
            mbar_init(&p_full[2 * i], 4);
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&o_done[i], 1);
            mbar_init(&h_done[i], 1);
            mbar_init(&last[i], 1);
        }
        mbar_init(q_full, PX_SOFT * 32);
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
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + L.slot);
    let_next_start();

    // Q, by the softmax warps: CH lanes of 16 bytes a row
    if (warp < PX_SOFT) {
        const int CH = D / 8;
        const int per = CH <= 8 ? 8 : CH <= 16 ? 16 : 32;  // lanes of a row
        const int c = lane & (per - 1);
        auto place = [&](int r) { return sm + ((r >> 7) * DB + (c >> 3)) * (PX_ROWS * 128) + swz(r & 127, c & 7); };
        const int rstep = PX_SOFT * 32 / per, db = rstep / a.G, dg = rstep - db * a.G;
        int b = (row0 + tid / per) / a.G, g = row0 + tid / per - b * a.G;  // of the next row
        auto next_source = [&]() {
            const uint16_t* const at = static_cast<const uint16_t*>(a.q) + b * a.q_sb + (kvh * a.G + g) * a.q_sh + c * 8;
            b += db, g += dg;
            if (g >= a.G) g -= a.G, ++b;
            return at;
        };
        if constexpr (E4 && QBF) {
#pragma unroll 8
            for (int r = tid / per; r < MT * PX_ROWS; r += rstep) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                const uint16_t* const from = next_source();
                if (row0 + r < R && c < CH) v = ld_128_l2(from);
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
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
                if (c < CH) *reinterpret_cast<uint4*>(place(r)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            mbar_arrive(q_full);
        } else {
            for (int r = tid / per; r < MT * PX_ROWS; r += rstep) {
                const bool have = row0 + r < R;
                const uint16_t* const from = next_source();
                if (c < CH) cp_async_16_zfill(place(r), have ? from : a.q, have ? 16 : 0);
            }
            arrive_after_copies(q_full);
        }
    }

    if (warp == PX_MMA) {
        const uint32_t lead = leader_lane();
        const uint32_t q0 = px_desc_lo(smem_addr(sm), 16), k0 = px_desc_lo(smem_addr(sm + L.k), 16),
                       v0 = px_desc_lo(smem_addr(sm + L.v), KT * 128);
        const uint32_t id_s = px_idesc(BF, false, KT), id_o = px_idesc(BF, true, D);
        const int nk = D / 16;
        bool ok = __all_sync(FULL_MASK, mbar_wait_abort(q_full, 0, abort));
        auto scores = [&](int j) {
            const int t = MT == 2 ? j >> 1 : j, st = t % KS;
            if (!__all_sync(FULL_MASK, mbar_wait_abort(&k_full[st], (t / KS) & 1, abort))) return false;
            fence_proxy_async();
            fence_after();
            const uint32_t q = q0 + (MT == 2 ? (j & 1) * (DB * PX_ROWS * 128 >> 4) : 0), k = k0 + st * (HALF >> 4);
            const uint32_t d = tmem + (j & 1) * 128;
#pragma unroll
            for (int kk = 0; kk < DB * 4; ++kk)
                if (kk < nk)
                    mma_ss(lead, d, q + (kk >> 2) * (PX_ROWS * 128 >> 4) + (kk & 3) * 2,
                           k + (kk >> 2) * (KT * 128 >> 4) + (kk & 3) * 2, id_s, kk > 0);
            mma_commit(lead, &s_full[j & 1]);
            if (lead) mbar_arrive(&s_full[j & 1]);
            if (MT == 1 || (j & 1)) mma_commit(lead, &k_empty[st]);
            return true;
        };
        for (int j = 0; j < 2 && j < jobs && ok; ++j) ok = scores(j);
        for (int j = 0; j < jobs && ok; ++j) {
            const int t = MT == 2 ? j >> 1 : j, st = t % VS, s = NS == 2 ? j & 1 : 0;
            if (!__all_sync(FULL_MASK, mbar_wait_abort(&v_full[st], (t / VS) & 1, abort))) {
                ok = false;
                break;
            }
            fence_proxy_async();
            const uint32_t o = tmem + 256 + s * 128, p = tmem + (j & 1) * 128, v = v0 + st * (HALF >> 4);
            const uint32_t more = j >= NS;
#pragma unroll
            for (int h = 0; h < 2 && ok; ++h) {
                ok = __all_sync(FULL_MASK, mbar_wait_abort(&p_full[2 * (j & 1) + h], (j >> 1) & 1, abort));
                if (!ok) break;
                fence_after();
#pragma unroll
                for (int kk = h * (KT / 32); kk < (h + 1) * (KT / 32); ++kk) {
                    const uint32_t pa = p + (kk >> 1) * 32 + (kk & 1) * 8;
                    mma_ts(lead, o, pa, v + kk * (2048 >> 4), id_o, kk > 0 ? 1u : more);
                    mma_ts(lead, o, pa + 16, v + kk * (2048 >> 4), id_o, 1u);
                }
                mma_commit(lead, h ? &o_done[s] : &h_done[s]);
            }
            if (!ok) break;
            if (j + NS >= jobs) mma_commit(lead, &last[s]);
            if (MT == 1 || (j & 1)) mma_commit(lead, &v_empty[st]);
            if (j + 2 < jobs) {  // into the buffer that PV(j) reads: not before it is done
                const int c = NS == 2 ? j >> 1 : j;
                ok = __all_sync(FULL_MASK, mbar_wait_abort(&o_done[s], c & 1, abort)) && scores(j + 2);
            }
        }
        // products already issued finish before tensor memory is freed
        mma_commit(lead, drained);
        mbar_wait(drained, 0);
    } else if (warp < PX_SOFT) {
        const int s = NS == 2 ? warp >> 2 : 0;
        const int r = (NS == 2 && MT == 2 ? s * PX_ROWS : 0) + (warp & 3) * 32 + lane;  // row of the group
        if (NS == 2 || warp < 4) {
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t o_at = tmem + lanes + 256 + s * 128;
            constexpr int HC = KT / 64;  // chunks of 32 keys in half a tile
            float m = -INFINITY;  // m: a whole number, so that its steps scale exactly
            float2 l2 = make_float2(0.f, 0.f);
            int c = 0;            // jobs of this stream so far
            bool ok = __all_sync(FULL_MASK, mbar_wait_abort(q_full, 0, abort));
            const bool flip = a.scale_log2 < 0.f;
            float sl = fabsf(a.scale_log2);
            if (E4 && QBF) sl *= back[r];
            sl = fmaxf(sl, 0x1p-126f);  // (masked scores of -inf stay so with a scale of 0)
            for (int j = s; j < jobs && ok; j += NS, ++c) {
                const int t = MT == 2 ? j >> 1 : j;
                ok = __all_sync(FULL_MASK, mbar_wait_abort(&s_full[j & 1], (j >> 1) & 1, abort));
                if (!ok) break;
                fence_after();
                const uint32_t s_at = tmem + lanes + (j & 1) * 128;
                const uint32_t* mask = live + (t % MASKS) * 4;
                // half of the tile's keys at a time become weights in their
                // place (a round trip to tensor memory, a maximum and a vote
                // take some 300 cycles whatever they are of)
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const uint32_t h_at = s_at + h * (KT / 2);
                    uint32_t x[HC][32];
#pragma unroll
                    for (int i = 0; i < HC; ++i) tm_ld32(h_at + i * 32, x[i]);
#pragma unroll
                    for (int i = 0; i < HC; ++i) tm_wait32(x[i]);
                    if (flip)
#pragma unroll
                        for (int i = 0; i < HC; ++i)
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[i][e] ^= 0x80000000u;
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < HC; ++i) {
                        const uint32_t on = mask[h * HC + i];
                        if (on != FULL_MASK)
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[i][e] = on >> e & 1u ? x[i][e] : 0xff800000u;
                        float m0 = __uint_as_float(x[i][0]), m1 = __uint_as_float(x[i][1]);
#pragma unroll
                        for (int e = 2; e < 30; e += 4) {
                            m0 = max3(m0, __uint_as_float(x[i][e]), __uint_as_float(x[i][e + 1]));
                            m1 = max3(m1, __uint_as_float(x[i][e + 2]), __uint_as_float(x[i][e + 3]));
                        }
                        m0 = max3(m0, __uint_as_float(x[i][30]), __uint_as_float(x[i][31]));
                        mx = max3(mx, m0, m1);
                    }
                    mx *= sl;
                    if (__any_sync(FULL_MASK, mx > m + SLACK)) {
                        // m moves up: so do l and O as far as it goes
                        const float mn = fmaxf(m, ceilf(mx));
                        const float f = exp2_ftz(m - finite_or_zero(mn));
                        m = mn;
                        l2.x *= f, l2.y *= f;
                        if (h || c > 0) {
                            // (phase by phase: a wait for one that comes after the next would
                            // pass at once.  S(c) was issued when PV(c - 2) of its stream, or
                            // a later one, was done)
                            if (c > 0) ok = ok && __all_sync(FULL_MASK, mbar_wait_abort(&o_done[s], (c - 1) & 1, abort));
                            if (h) ok = ok && __all_sync(FULL_MASK, mbar_wait_abort(&h_done[s], c & 1, abort));
                            fence_after();
                            for (int d = 0; d < D; d += 16) {
                                uint32_t w[16];
                                tm_ld16(o_at + d, w);
#pragma unroll
                                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
                                tm_st16(o_at + d, w);
                            }
                        }
                    }
                    const float mu = finite_or_zero(m) - P_SHIFT;
                    const float2 sl2 = make_float2(sl, sl), mu2 = make_float2(-mu, -mu);
#pragma unroll
                    for (int i = 0; i < HC; ++i) {
                        uint32_t w[32];  // hi, then lo
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 p = __ffma2_rn(make_float2(__uint_as_float(x[i][2 * e]), __uint_as_float(x[i][2 * e + 1])), sl2, mu2);
                            p = make_float2(exp2_ftz(p.x), exp2_ftz(p.y));
                            l2 = __fadd2_rn(l2, p);
                            w[e] = pack2<BF>(p.x, p.y);
                            const float2 r = rest2<BF>(p, w[e]);
                            w[16 + e] = pack2<BF>(r.x, r.y);
                        }
                        tm_st32(h_at + i * 32, w);
                    }
                    wait_st();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * (j & 1) + h]);
                }
            }
            const float l = l2.x + l2.y;
            // the piece: (m, l) and O of this row, O only where some job ran
            if (ok && c > 0) ok = __all_sync(FULL_MASK, mbar_wait_abort(&last[s], 0, abort));
            const int row = row0 + r;
            const int piece = MT == 1 && NS == 2 ? 2 * split + s : split;
            const int64_t at = ((int64_t)kvh * a.pieces + piece) * R + row;
            if (row < R)
                reinterpret_cast<float2*>(a.ws_ml)[at] = ok && c > 0 ? make_float2(m - P_SHIFT, l) : make_float2(-INFINITY, 0.f);
            if (ok && c > 0) {
                fence_after();
                float* out = a.ws_o + at * D;
                // (32 rows of 32 bytes are 32 lines to the load-store unit; four
                // lanes exchange their blocks and write one row's 128 bytes)
                const int lane0 = row - (lane & 3);
                for (int d = 0; d < D; d += 32) {
                    uint32_t o[32];
                    if (d + 32 <= D) {
                        tm_ld32(o_at + d, o);
                        tm_wait32(o);
                    } else {
                        uint32_t u[16];
                        tm_ld16(o_at + d, u);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = u[e], o[16 + e] = 0u;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        exchange(o[e], o[8 + e], lane & 1, 1);
                        exchange(o[16 + e], o[24 + e], lane & 1, 1);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        exchange(o[e], o[16 + e], lane & 2, 2);
                        exchange(o[8 + e], o[24 + e], lane & 2, 2);
                    }
                    // block n is now row lane0 + n's dims d + 8 (lane & 3) ..
                    const int dim = d + 8 * (lane & 3);
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        if (lane0 + n < R && dim < D)
                            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out + (n - (lane & 3)) * D + dim),
                                         "r"(o[8 * n]), "r"(o[8 * n + 1]), "r"(o[8 * n + 2]), "r"(o[8 * n + 3]),
                                         "r"(o[8 * n + 4]), "r"(o[8 * n + 5]), "r"(o[8 * n + 6]), "r"(o[8 * n + 7])
                                         : "memory");
                }
            }
        }
    } else {
        // ---------------- K and V tiles, two warps each ----------------
        const bool is_v = warp >= PX_VW;
        const int pt = tid - (is_v ? PX_VW : PX_KW) * 32;  // 0 .. 63
        uint64_t* const full = is_v ? v_full : k_full;
        uint64_t* const empty = is_v ? v_empty : k_empty;
        uint8_t* const ring = sm + (is_v ? L.v : L.k);
        constexpr int ES = E4 ? 1 : 2;
        const int stages = KS == VS ? KS : is_v ? VS : KS;
        const int64_t sp = (is_v ? a.v_sp : a.k_sp) * ES, stt = (is_v ? a.v_st : a.k_st) * ES;
        const uint8_t* const src = static_cast<const uint8_t*>(is_v ? a.v : a.k) + (int64_t)kvh * (is_v ? a.v_sh : a.k_sh) * ES;

        // The places of the next pages, so that no tile waits for a lookup: a
        // window of the page table that moves on when a tile passes its end.
        // (Reading the rows' places below has no branch: all at once.)
        constexpr int64_t NONE = INT64_MIN;
        int64_t* const places = reinterpret_cast<int64_t*>(sm + L.pages) + (is_v ? PX_PAGES : 0);
        auto page_of = [&](int key) { return (int)(((uint64_t)(uint32_t)key * a.page_mul) >> a.page_shift); };
        const int key0 = tile0 * KT, key_end = min((tile0 + tiles) * KT, a.len), last_page = page_of(key_end - 1);
        int page0 = 0, held_to = -1;  // pages page0 .. held_to
        auto together = [&]() {
            if (is_v)
                asm volatile("bar.sync 2, %0;" ::"n"(PX_BRING) : "memory");
            else
                asm volatile("bar.sync 1, %0;" ::"n"(PX_BRING) : "memory");
        };
        auto hold_pages = [&](int t) {  // those of tile t
            const int first = key0 + t * KT;
            if (page_of(min(first + KT, key_end) - 1) <= held_to) return;
            together();
            page0 = page_of(first);
            held_to = min(page0 + PX_PAGES - 1, last_page);
            for (int i = page0 + pt; i <= held_to; i += PX_BRING) {
                const int pg = __ldcg(a.table + i);
                const bool known = pg >= 0 && pg < a.num_pages;
                if (!known) atomicOr(a.err, MOE_DEVERR_PAGE);
                places[i - page0] = known ? pg * sp : NONE;
            }
            together();
        };
        auto place_of = [&](int key) {  // bytes from the head's first row; NONE behind the end
            const int pi = page_of(min(key, key_end - 1));
            const int64_t at = places[pi - page0];
            const int64_t row = at + (int64_t)((uint64_t)(uint32_t)(key - pi * a.page) * (uint64_t)stt);
            return key < key_end && at != NONE ? row : NONE;
        };
        // Tile t's rows, found once for the lanes that share them; and by the K
        // warps the masks of those that are live.
        int64_t* const rows_of = reinterpret_cast<int64_t*>(sm + L.rows) + (is_v ? 256 : 0);
        auto find_rows = [&](int t) {
            hold_pages(t);
#pragma unroll
            for (int i = 0; i < KT / PX_BRING; ++i) {
                const int key = i * PX_BRING + pt;
                const int64_t at = place_of(key0 + t * KT + key);
                rows_of[(t & 1) * 128 + key] = at;
                if (!is_v) {
                    const uint32_t word = __ballot_sync(FULL_MASK, at != NONE);
                    if (lane == 0) live[(t % MASKS) * 4 + (key >> 5)] = word;
                }
            }
            together();
        };
        // `whole`: the head fills its blocks of 64 dims (D = 64 DB), so that the
        // steps from a thread's piece to its next are constants.
        auto bring = [&](auto whole) {
            constexpr bool W = decltype(whole)::value;
            bool ok = true;
            if constexpr (!E4) {
                const int CH = W ? DB * 8 : D / 8, per = PX_BRING / CH;  // rows that the two warps copy at once
                const int c = pt % CH, r0 = pt / CH;
                const uint32_t col = (c >> 3) * (KT * 128);
                const uint8_t* const from = src + c * 16;
                for (int t = 0; t < tiles; ++t) {
                    const int st = t % stages;
                    find_rows(t);
                    if (t >= stages && ok) ok = __all_sync(FULL_MASK, mbar_wait_abort(&empty[st], ((t / stages) - 1) & 1, abort));
                    if (!ok) continue;  // (the two warps stay together in find_rows)
                    uint8_t* const dst = ring + st * HALF + col;
                    const int64_t* const o = rows_of + (t & 1) * 128 + r0;
                    // (eight rows' places are read before their copies, which
                    // order the accesses to shared memory around them)
                    if (W || r0 < per)
#pragma unroll 1
                        for (int row = 0; row < KT; row += 8 * per) {
                            int64_t at[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) at[i] = o[W ? row + i * per : min(row + i * per, KT - 1 - r0)];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (W || r0 + row + i * per < KT)
                                    cp_async_16_zfill(dst + swz(r0 + row + i * per, c & 7), at[i] == NONE ? from : from + at[i],
                                                      at[i] == NONE ? 0 : 16);
                        }
                    arrive_after_copies(&full[st]);
                    if (!is_v && lane == 0) mbar_arrive(&full[st]);  // (carries the masks)
                }
            } else {
                // 16 codes at a time; a thread widens the pieces that it has
                // copied itself, and piece i of all threads lies together.  Of a
                // whole head eight lanes take 4 pieces of each of two rows, so
                // that they write the 8 different 16-byte columns of the swizzle;
                // else they go row by row.
                constexpr int PER = KT * DB * 4 / PX_BRING;  // pieces of a thread at most
                constexpr int KC = px_k_codes(DB, E4), VC = px_v_codes(DB, E4);
                const int ahead = KC == VC ? KC : is_v ? VC : KC;
                constexpr int BATCH = PER < 8 ? PER : 8;  // pieces that are read before any of them is written
                uint8_t* const codes = sm + L.codes + (is_v ? KC * (HALF / 2) : 0) + pt * 16;
                const int CH = W ? DB * 4 : D / 16, unit = pt >> 3;
                const int row0 = W ? 2 * (unit / DB) + (pt >> 2 & 1) : pt / CH, c0 = W ? 4 * (unit % DB) + (pt & 3) : pt % CH;
                const int dr = W ? 16 / DB : PX_BRING / CH, dc = W ? 0 : PX_BRING % CH;
                auto step = [&](int& row, int& c) {  // to the thread's next piece
                    row += dr;
                    if (!W) {
                        c += dc;
                        if (c >= CH) c -= CH, ++row;
                    }
                };
                auto copy = [&](int t) {
                    if (t < tiles) {
                        find_rows(t);
                        const int64_t* const o = rows_of + (t & 1) * 128;
                        uint8_t* const to = codes + (t % ahead) * (HALF / 2);
                        int row = row0, c = c0;
                        if (!W) asm volatile("" : "+r"(row), "+r"(c));  // (16 pieces' steps are not worth registers)
#pragma unroll
                        for (int i0 = 0; i0 < PER; i0 += BATCH) {
                            int64_t at[BATCH];  // (as above)
#pragma unroll
                            for (int i = 0; i < BATCH; ++i) {
                                at[i] = o[W ? row : min(row, KT - 1)];
                                if (!W) at[i] = row < KT && at[i] != NONE ? at[i] + c * 16 : NONE;
                                step(row, c);
                            }
#pragma unroll
                            for (int i = 0; i < BATCH; ++i)
                                cp_async_16_zfill(to + (i0 + i) * (PX_BRING * 16),
                                                  (at[i] == NONE ? src : src + at[i]) + (W ? c0 * 16 : 0), at[i] == NONE ? 0 : 16);
                        }
                    }
                    cp_async_commit();
                };
#pragma unroll 1
                for (int t = 0; t < ahead; ++t) copy(t);
                for (int t = 0; t < tiles; ++t) {
                    const int st = t % stages;
                    if (KC == VC || !is_v)
                        cp_async_wait<KC - 1>();
                    else
                        cp_async_wait<VC - 1>();
                    if (t >= stages && ok) ok = __all_sync(FULL_MASK, mbar_wait_abort(&empty[st], ((t / stages) - 1) & 1, abort));
                    if (!ok) {
                        copy(t + ahead);  // (as above)
                        continue;
                    }
                    const uint8_t* const from = codes + (t % ahead) * (HALF / 2);
                    uint8_t* const dst = ring + st * HALF;
                    int row = row0, c = c0;
                    if (!W) asm volatile("" : "+r"(row), "+r"(c));
#pragma unroll
                    for (int i0 = 0; i0 < PER; i0 += BATCH) {
                        uint4 x[BATCH];
#pragma unroll
                        for (int i = 0; i < BATCH; ++i) x[i] = *reinterpret_cast<const uint4*>(from + (i0 + i) * (PX_BRING * 16));
#pragma unroll
                        for (int i = 0; i < BATCH; ++i) {
                            uint32_t w[8];
                            e4m3x4_to_f16(x[i].x, w[0], w[1]);
                            e4m3x4_to_f16(x[i].y, w[2], w[3]);
                            e4m3x4_to_f16(x[i].z, w[4], w[5]);
                            e4m3x4_to_f16(x[i].w, w[6], w[7]);
                            if (W || row < KT) {
                                uint8_t* const d = dst + (c >> 2) * (KT * 128);
                                *reinterpret_cast<uint4*>(d + swz(row, (2 * c) & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
                                *reinterpret_cast<uint4*>(d + swz(row, (2 * c + 1) & 7)) = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                            step(row, c);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[st]);
                    copy(t + ahead);
                }
            }
        };
        if (D == DB * 64)
            bring(std::true_type{});
        else
            bring(std::false_type{});
    }
    cp_async_commit();
    cp_async_wait<0>();  // no copy still in flight on any exit
    fence_before();
    __syncthreads();
    if (warp == PX_MMA) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
    if (tid == 0 && *abort) atomicOr(a.err, MOE_DEVERR_TIMEOUT);
    after_previous();
}

// Every output from its pieces: the sequence's own and, where it shares the
// prefix, the prefix's.  A thread takes four dims of a row, and a.join_groups
// threads with the same dims divide the row's pieces between them, four or so
// each with all loads in flight; the groups are added in order.  A piece whose
// weights are all 0 is left out (its sums may hold anything); one whose scores
// are all NaN has no maximum either, but a sum of NaN, which has to show.
constexpr int PJ_THREADS = 256, PJ_FLIGHT = 4, PJ_BLOCKS = 5;  // (blocks of an SM)
template <bool QBF>
__global__ void __launch_bounds__(PJ_THREADS, PJ_BLOCKS) prefix_join_kernel(const __grid_constant__ PrefixArgs a) {
    __shared__ float4 sm_o[PJ_THREADS];
    __shared__ float2 sm_ml[PJ_THREADS];
    const int vecs = a.D / 4, per_row = vecs * a.join_groups;
    const int slot = threadIdx.x / per_row, in_row = threadIdx.x - slot * per_row;
    const int g = in_row / vecs, dim = (in_row - g * vecs) * 4;
    const int64_t bh = (int64_t)blockIdx.x * (PJ_THREADS / per_row) + slot;
    const bool on = slot < PJ_THREADS / per_row && bh < (int64_t)a.B * a.Hq;
    const int b = on ? (int)(bh / a.Hq) : 0, h = on ? (int)(bh - (int64_t)b * a.Hq) : 0;
    const int kvh = h / a.G, R = a.B * a.G, row = b * a.G + (h - kvh * a.G);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    auto scale = [&](float mn) {
        const float old = exp2_ftz(m - finite_or_zero(mn));
        m = mn;
        l *= old;
        sum.x *= old, sum.y *= old, sum.z *= old, sum.w *= old;
    };
    auto add = [&](float2 ml, const float4& v) {
        if (ml.x == -INFINITY && ml.y == 0.f) return;
        const float f = exp2_ftz(ml.x - finite_or_zero(m));
        l += f * ml.y;
        sum.x += f * v.x, sum.y += f * v.y, sum.z += f * v.z, sum.w += f * v.w;
    };
    after_previous();
    if (on) {
        int np = 0;
        if (min((int64_t)a.lens[b], a.cap) >= a.len && (!a.shares || a.shares[b])) {
            const int g0 = row / a.group_rows * a.group_rows;
            np = a.group_rows > PX_ROWS && R - g0 <= PX_ROWS ? 2 * a.splits : a.splits;
        }
        const float2* const mls = reinterpret_cast<const float2*>(a.ws_ml) + (int64_t)kvh * a.pieces * R + row;
        const float* const os = a.ws_o + ((int64_t)kvh * a.pieces * R + row) * a.D + dim;
        float2 own_ml = make_float2(-INFINITY, 0.f);
        float4 own = make_float4(0.f, 0.f, 0.f, 0.f);
        if (g == 0) {
            own_ml = reinterpret_cast<const float2*>(a.own_ml)[bh];
            own = *reinterpret_cast<const float4*>(a.own_o + bh * a.D + dim);
        }
#pragma unroll 1
        for (int p0 = g; p0 < np; p0 += PJ_FLIGHT * a.join_groups) {
            float4 v[PJ_FLIGHT];
            float2 ml[PJ_FLIGHT];
#pragma unroll
            for (int i = 0; i < PJ_FLIGHT; ++i) {
                const int p = p0 + i * a.join_groups;
                ml[i] = make_float2(-INFINITY, 0.f);
                if (p < np) {
                    ml[i] = mls[(int64_t)p * R];
                    v[i] = *reinterpret_cast<const float4*>(os + (int64_t)p * R * a.D);
                }
            }
            float mn = m;
#pragma unroll
            for (int i = 0; i < PJ_FLIGHT; ++i) mn = fmaxf(mn, ml[i].x);
            scale(mn);
#pragma unroll
            for (int i = 0; i < PJ_FLIGHT; ++i)
                if (p0 + i * a.join_groups < np) add(ml[i], v[i]);
        }
        if (g == 0) {
            scale(fmaxf(m, own_ml.x));
            add(own_ml, own);
        }
    }
    if (a.join_groups > 1) {  // (the same in all threads)
        sm_ml[threadIdx.x] = make_float2(m, l);
        sm_o[threadIdx.x] = sum;
        __syncthreads();
        if (on && g == 0) {
            float mn = m;
            for (int i = 1; i < a.join_groups; ++i) mn = fmaxf(mn, sm_ml[threadIdx.x + i * vecs].x);
            scale(mn);
            for (int i = 1; i < a.join_groups; ++i) add(sm_ml[threadIdx.x + i * vecs], sm_o[threadIdx.x + i * vecs]);
        }
    }
    if (!on || g > 0) return;
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

// Whether the prefix is worth its own launch and the join: reading it by each
// sequence costs (B - 1) more times its keys and values, the three launches and
// the pieces some 3 to 10 us.  Measured (us, this form / one launch of the paged
// kernel, * what is taken, B sequences with 60 own tokens, which all share; the
// flags are on the device, so sequences that do not share count like the others):
//   32 / 4 heads of 128, BF16: 128 x 128 18.2 / 12.6*, 8 x 512 10.8 / 11.5*, 32 x 512
//     13.6* / 13.1, 8 x 4096 16.6* / 19.3, 64 x 4096 23.6* / 49.6, 2 x 16384 18.0* / 19.1
//   8 / 8 of 64, FP16: 16 x 512 11.7 / 9.5*, 32 x 512 12.5* / 12.9, 64 x 512 13.0* / 17.4
//   32 / 4 of 128, E4M3, BF16 query: 64 x 512 21.6 / 18.3*, 8 x 4096 18.4 / 18.1*,
//     4 x 16384 20.6* / 23.1, 8 x 8192 20.3* / 22.8, 64 x 1024 23.4* / 22.9, 32 x 4096
//     24.9* / 28.9, 2 x 65536 40.8 / 30.3*, 3 x 65536 41.1 / 38.3*; FP16 query: 4 x 16384
//     19.7* / 22.2, 64 x 1024 18.6* / 22.2, 4 x 32768 27.4* / 30.3, 3 x 65536 39.5 / 37.5*
//   other sizes, E4M3, FP16 query: 8 / 8 of 64, 8 x 8192 16.7* / 22.0; 64 / 8 of 128,
//     8 x 2048 16.0 / 14.4*, 4 x 8192 20.2* / 21.9; 12 / 12 of 80, 7 x 5016 24.4 / 22.7*,
//     20 x 2508 20.7* / 30.7; of 192, 8 x 2048 21.2 / 19.6*, 32 x 512 18.1* / 23.0;
//     16 / 4 of 256, 16 x 2048 17.7 / 17.0*
// so by what is saved, from four key tiles on; codes have to be widened first,
// which the paged kernel does on its way: they take more, most where a head does
// not fill its blocks of 64 dims or two streams (D = 64 and 128 do), and four
// sequences.
bool prefix_pays(int B, int Hkv, int D, int len, bool e4) {
    const double saved = 2.0 * (B - 1) * len * Hkv * D;  // elements
    if (len < 512) return false;
    if (!e4) return saved >= 12e6;
    return B >= 4 && saved >= (D == 64 || D == 128 ? 48e6 : 70e6);
}

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
    constexpr size_t smem = px_layout(DB, KV == KV_E4M3).total + 1024;
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
    // (threads beyond what is resident at once would take another round: without
    // that limit 32 x 8192 tokens take 31.3 us in place of 29.4, 64 x 65536 five more)
    const int np = a.B * a.G <= PX_ROWS ? a.pieces : a.splits, vecs = a.D / 4;
    const int64_t resident = (int64_t)di.sm_count * PJ_BLOCKS * PJ_THREADS;
    a.join_groups = 1;
    while (a.join_groups * PJ_FLIGHT < np && 2 * a.join_groups * vecs <= PJ_THREADS &&
           2 * a.join_groups * (int64_t)vecs * (int64_t)rows <= resident)
        a.join_groups *= 2;
    const int per_block = PJ_THREADS / (vecs * a.join_groups);
    const dim3 blocks((unsigned)((rows + per_block - 1) / per_block));
    return dtype == MOE_BF16 ? launch_after(prefix_join_kernel<true>, blocks, PJ_THREADS, 0, st, a)
                             : launch_after(prefix_join_kernel<false>, blocks, PJ_THREADS, 0, st, a);
}

}  // namespace moedec
