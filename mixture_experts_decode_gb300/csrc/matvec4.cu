// matvec4.cu -- products of 4-bit weights with few activation rows.
//
// Mathematics.  With unsigned codes c, zero points z (8 where none are given)
// and scales s per row n and group g of consecutive k:
//   y[t,n] = sum_g s[n,g] * ( sum_{k in g} c[n,k] x[t,k] - z[n,g] sum_{k in g} x[t,k] ).
// A code becomes the 16-bit float 16 + c by placing its four bits at the top
// of the mantissa of 16.0 (one shift, one logic operation per pair of codes;
// exact in BF16 and FP16), and the sum of x over the group comes from the same
// matrix instruction with a row of ones, so the group's part is
//   s * ( sum (16 + c) x - (16 + z) sum x ),
// products exact, sums FP32.  The offset makes the two sums about five times
// larger than their difference for spread codes, which costs two or three of
// FP32's bits; the weights themselves are never rounded.  (One row of x on many
// weight rows: products of 8-bit parts of x, to the same accuracy, below.)
//
// Bound: HBM on the codes for few rows of x (half a byte per weight; scales
// and zero points add 3 bytes per group), then instruction issue: about 26
// instructions per eight codes of a thread, all told (28672 x 8192, one row:
// 129 MB in 34.7 us, 3.7 TB/s, 2.5 instructions per cycle of 4).  A warp takes 16 * MT weight rows
// (M of mma.m16n8k16) by 256 k per step through its own cp.async ring, eight
// rows of x are the N side, and the eight warps of a block split K, so a
// single token still has every warp of the GPU loading; their sums meet in
// shared memory once per tile, and blocks stride over the tiles with the ring
// running on across them.
#include <algorithm>

#include "block_common.cuh"
#include "internal.h"

namespace moedec {

namespace {

constexpr int MV_WARPS = 8;
constexpr int MV_STEP = 256;           // k per step
constexpr int MV_ROW = MV_STEP / 2;    // bytes of a row's step

template <bool BF>
__device__ __forceinline__ void mv_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with a sum of zero to begin with.
template <bool BF>
__device__ __forceinline__ void mv_mma0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Codes I and I + 4 of a word as the pair 16 + c (I = 0..3): the nibbles of
// the two 16-bit halves moved to the mantissa's top four bits.
template <bool BF, int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    constexpr int TOP = BF ? 3 : 6;  // lowest of the mantissa's top four bits
    constexpr int SH = 4 * I - TOP;
    const uint32_t v = SH >= 0 ? w >> (SH >= 0 ? SH : 0) : w << (SH < 0 ? -SH : 0);
    return (v & (0x000f000fu << TOP)) | (BF ? 0x41804180u : 0x4c004c00u);
}

// Stages of a warp's ring, blocks of 32 k whose x is loaded together, and
// blocks per SM that the registers are cut for.
constexpr int mv_stages(int mt) { return mt == 1 ? 4 : 3; }
constexpr int mv_ahead(int nt) { return nt == 1 ? 8 : nt == 2 ? 4 : 2; }
constexpr int mv_blocks(int nt) { return nt <= 2 ? 2 : 1; }

// ---- E4M3 products (few rows of x) ----

template <bool BF>
__device__ __forceinline__ void x_floats(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 p;
        if (BF) {
            p = bf16x2_to_float2(w[i]);
        } else {
            __half2 h;
            memcpy(&h, &w[i], 4);
            p = __half22float2(h);
        }
        f[2 * i] = p.x, f[2 * i + 1] = p.y;
    }
}
// Four floats -> four E4M3 codes, a in the lowest byte.
__device__ __forceinline__ uint32_t e4m3_four(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | (uint32_t)hi << 16;
}
// Exponent e of a group's largest element, 2^e <= amax < 2^(e + 1), within what
// keeps 2^(7 - e) and its inverse normal numbers (128 for an infinity or NaN).
__device__ __forceinline__ int x_exponent(uint32_t amax) { return max((int)(amax >> 23) - 127, -112); }

__device__ __forceinline__ void e4m3_mma(float (&c)[4], const uint32_t (&a)[4], uint2 b, bool first) {
    if (first)
        asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(0.f));
    else
        asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
constexpr int MV_ONE_STAGES = 2;
constexpr int MV_PARTS = 3;

}  // namespace

// GB: blocks of 32 k per group (1, 2, 4).
template <int MT, int NT, int GB, bool BF>
__global__ void __launch_bounds__(MV_WARPS * 32, mv_blocks(NT)) matvec4_kernel(const __grid_constant__ Matvec4Args a, int tiles, int steps, int kw_log) {
    constexpr int NST = mv_stages(MT);
    constexpr int STAGE = MT * 16 * MV_ROW;
    constexpr int NGS = 8 / GB;              // groups of a step
    constexpr int W = mv_ahead(NT);
    constexpr int OUT = MT * NT * 4;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_index();
    const int g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * NST * STAGE;
    float* sm_sum = reinterpret_cast<float*>(smem + MV_WARPS * NST * STAGE);  // [warps][OUT][32]
    const int tok0 = blockIdx.y * (NT * 8);
    const int toks = min(a.T - tok0, NT * 8);
    after_previous();
    const int kg = a.K / a.group;
    // 2^kw_log warps share K (step = i * that + kw), the others take further rows
    const int kws = 1 << kw_log, kw = warp & (kws - 1), rw = warp >> kw_log;
    const int tile_rows = (MV_WARPS >> kw_log) * (MT * 16);
    const int per_warp = (steps + kws - 1) >> kw_log;  // steps of a warp and tile
    const int my_tiles = ((int)blockIdx.x < tiles) ? (tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    // Rows beyond T read the first row of x again: their columns of the
    // products are not stored, and no column depends on another.
    const uint16_t* xrow[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int tk = nt * 8 + g;
        xrow[nt] = static_cast<const uint16_t*>(a.x) + (int64_t)(tok0 + (tk < toks ? tk : 0)) * a.x_stride;
    }

    // Nothing below branches per lane, because the matrix instructions need
    // the whole warp together: weight rows beyond N read the last row again
    // (not stored), columns beyond K the last ones (their scale is zero).
    // The pipeline runs over (tile, step) pairs, issue side and use side.
    const int64_t row_bytes = a.K / 2;
    const int last_kb = a.K / 2 - 16;
    int is_tile = 0, is_step = 0, is_stage = 0;
    auto issue = [&]() {
        if (is_tile < my_tiles) {
            const int64_t row0 = (int64_t)(blockIdx.x + (int64_t)is_tile * gridDim.x) * tile_rows + rw * (MT * 16);
            const int r = lane >> 3;
            const int kb = min((is_step * kws + kw) * MV_ROW + (lane & 7) * 16, last_kb);
            uint8_t* s = ring + is_stage * STAGE + r * MV_ROW;
            const int sw0 = ((lane & 7) ^ r) << 4, sw1 = sw0 ^ 64;  // row & 7 is r or r + 4
            if (row0 + MT * 16 <= a.N) {
                const uint8_t* p = a.codes + (row0 + r) * row_bytes + kb;
#pragma unroll
                for (int i = 0; i < MT * 4; ++i, p += 4 * row_bytes)
                    cp_async_16_zfill(s + i * 4 * MV_ROW + (i & 1 ? sw1 : sw0), p, 16);
            } else {
#pragma unroll
                for (int i = 0; i < MT * 4; ++i)
                    cp_async_16_zfill(s + i * 4 * MV_ROW + (i & 1 ? sw1 : sw0),
                                      a.codes + min(row0 + r + i * 4, (int64_t)a.N - 1) * row_bytes + kb, 16);
            }
            if (++is_step == per_warp) {
                is_step = 0;
                ++is_tile;
            }
            if (++is_stage == NST) is_stage = 0;
        }
        cp_async_commit();
    };
    // Scales (in pairs) and zeros (in fours) of a step's groups for one row per
    // lane (MT = 1: twice), loaded a step ahead and not touched until then.
    uint32_t sc[(NGS + 1) / 2], zb[(NGS + 3) / 4];
    int sz_tile = 0, sz_step = 0;
    const bool whole_groups = kg % NGS == 0 && a.scales_aligned;
    auto fetch_sz = [&]() {
        const int64_t row = min((int64_t)(blockIdx.x + (int64_t)sz_tile * gridDim.x) * tile_rows + rw * (MT * 16) + (lane & (MT * 16 - 1)),
                                (int64_t)a.N - 1);
        const int gi0 = (sz_step * kws + kw) * NGS;
        if (whole_groups && gi0 < kg) {
            const int64_t at = row * kg + gi0;
            const uint16_t* sp = static_cast<const uint16_t*>(a.scales) + at;
            if constexpr (NGS == 8) {
                const uint4 v = *reinterpret_cast<const uint4*>(sp);
                sc[0] = v.x, sc[1] = v.y, sc[2] = v.z, sc[3] = v.w;
                const uint2 z = a.zeros ? *reinterpret_cast<const uint2*>(a.zeros + at) : make_uint2(0x08080808u, 0x08080808u);
                zb[0] = z.x, zb[1] = z.y;
            } else if constexpr (NGS == 4) {
                const uint2 v = *reinterpret_cast<const uint2*>(sp);
                sc[0] = v.x, sc[1] = v.y;
                zb[0] = a.zeros ? *reinterpret_cast<const uint32_t*>(a.zeros + at) : 0x08080808u;
            } else {
                sc[0] = *reinterpret_cast<const uint32_t*>(sp);
                zb[0] = a.zeros ? *reinterpret_cast<const uint16_t*>(a.zeros + at) : 0x0808u;
            }
        } else {  // one by one; groups beyond K get scale 0
#pragma unroll
            for (int i = 0; i < (NGS + 3) / 4; ++i) zb[i] = 0;
#pragma unroll
            for (int i = 0; i < NGS; ++i) {
                const int gi = min(gi0 + i, kg - 1);
                uint32_t v = static_cast<const uint16_t*>(a.scales)[row * kg + gi];
                v = gi0 + i < kg ? v : 0u;
                sc[i / 2] = i % 2 ? sc[i / 2] | v << 16 : v;
                zb[i / 4] |= (a.zeros ? (uint32_t)a.zeros[row * kg + gi] : 8u) << (8 * (i % 4));
            }
        }
        if (++sz_step == per_warp) {
            sz_step = 0;
            ++sz_tile;
        }
    };
#pragma unroll 1
    for (int i = 0; i < NST - 1; ++i) issue();
    fetch_sz();

    int use_stage = 0;
    for (int tile = 0; tile < my_tiles; ++tile) {
        const int64_t row0 = (int64_t)(blockIdx.x + (int64_t)tile * gridDim.x) * tile_rows;
        float tot[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) tot[mt][nt][j] = 0.f;

#pragma unroll 1
        for (int si = 0; si < per_warp; ++si) {
            const int step = si * kws + kw;
            uint32_t sz[NGS];  // scale | FP16 of 16 + zero << 16
            // 1024 + z by its bits, less 1008: 16 + z, exact
#pragma unroll
            for (int i = 0; i < NGS / 2; ++i) {
                const uint32_t zp = __byte_perm(zb[i / 2], 0u, i % 2 ? 0x4342 : 0x4140) | 0x64006400u;
                uint32_t zz;
                asm("sub.f16x2 %0, %1, %2;" : "=r"(zz) : "r"(zp), "r"(0x63e063e0u));
                sz[2 * i] = __byte_perm(sc[i], zz, 0x5410);
                sz[2 * i + 1] = __byte_perm(sc[i], zz, 0x7632);
            }
            // x of the first blocks (L1 or L2), under the wait for the codes
            uint4 xv[W][NT];
            auto load_x = [&](int blk0) {
#pragma unroll
                for (int i = 0; i < W; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        xv[i][nt] = ld_128(xrow[nt] + min(step * MV_STEP + (blk0 + i) * 32 + 8 * t, a.K - 8));
            };
            load_x(0);
            cp_async_wait<NST - 2>();
            __syncwarp();
            issue();
            fetch_sz();
            const uint8_t* s = ring + use_stage * STAGE;
            if (++use_stage == NST) use_stage = 0;
#pragma unroll
            for (int grp = 0; grp < NGS; ++grp) {
                float acc[MT][NT][4], xs[NT][4];
#pragma unroll
                for (int bb = 0; bb < GB; ++bb) {
                    const int blk = grp * GB + bb;
                    if (blk && blk % W == 0) load_x(blk);
                    uint32_t xb[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 v = xv[blk % W][nt];
                        xb[nt][0] = __byte_perm(v.x, v.z, 0x5410);  // x0, x4
                        xb[nt][1] = __byte_perm(v.x, v.z, 0x7632);  // x1, x5
                        xb[nt][2] = __byte_perm(v.y, v.w, 0x5410);  // x2, x6
                        xb[nt][3] = __byte_perm(v.y, v.w, 0x7632);  // x3, x7
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const int sw = ((blk ^ g) << 4) + 4 * t;
                        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(s + (mt * 16 + g) * MV_ROW + sw);
                        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(s + (mt * 16 + g + 8) * MV_ROW + sw);
                        const uint32_t a0[4] = {code_pair<BF, 0>(w0), code_pair<BF, 0>(w1), code_pair<BF, 1>(w0),
                                                code_pair<BF, 1>(w1)};
                        const uint32_t a1[4] = {code_pair<BF, 2>(w0), code_pair<BF, 2>(w1), code_pair<BF, 3>(w0),
                                                code_pair<BF, 3>(w1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (bb == 0)
                                mv_mma0<BF>(acc[mt][nt], a0, xb[nt][0], xb[nt][1]);
                            else
                                mv_mma<BF>(acc[mt][nt], a0, xb[nt][0], xb[nt][1]);
                            mv_mma<BF>(acc[mt][nt], a1, xb[nt][2], xb[nt][3]);
                        }
                    }
                    constexpr uint32_t one = BF ? 0x3f803f80u : 0x3c003c00u;
                    const uint32_t ones[4] = {one, one, one, one};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (bb == 0)
                            mv_mma0<BF>(xs[nt], ones, xb[nt][0], xb[nt][1]);
                        else
                            mv_mma<BF>(xs[nt], ones, xb[nt][0], xb[nt][1]);
                        mv_mma<BF>(xs[nt], ones, xb[nt][2], xb[nt][3]);
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t v = __shfl_sync(FULL_MASK, sz[grp], mt * 16 + h * 8 + g);
                        float sc;
                        if (BF) {
                            sc = __uint_as_float(v << 16);
                        } else {
                            __half hh;
                            const uint16_t q = (uint16_t)v;
                            memcpy(&hh, &q, 2);
                            sc = __half2float(hh);
                        }
                        const float zz = __half2float(__ushort_as_half((uint16_t)(v >> 16)));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                tot[mt][nt][2 * h + c] +=
                                    sc * fmaf(-zz, xs[nt][c], acc[mt][nt][2 * h + c]);
                    }
            }
        }

        // the warps' sums, in their order
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) sm_sum[(warp * OUT + (mt * NT + nt) * 4 + j) * 32 + lane] = tot[mt][nt][j];
        __syncthreads();
        // consecutive threads take consecutive rows of a token
        for (int e = tid; e < tile_rows * toks; e += MV_WARPS * 32) {
            const int tk = e / tile_rows, r = e - tk * tile_rows;
            const int mt = (r >> 4) % MT, rg = r & 7, h = (r >> 3) & 1;
            const int nt = tk >> 3, tt = (tk & 7) >> 1, c = tk & 1;
            const int at = ((mt * NT + nt) * 4 + 2 * h + c) * 32 + rg * 4 + tt;
            const float* first = sm_sum + ((r / (MT * 16)) << kw_log) * OUT * 32 + at;
            float v = 0.f;
            for (int w = 0; w < kws; ++w) v += first[w * OUT * 32];
            const int64_t row = row0 + r;
            if (row < a.N) {
                const int64_t o = (int64_t)(tok0 + tk) * a.y_stride + row;
                if (BF)
                    static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(v);
                else
                    static_cast<__half*>(a.y)[o] = __float2half_rn(v);
            }
        }
        __syncthreads();
    }
    cp_async_wait<0>();
}

// One row of x, many of weights: the products in E4M3.  GB as above.
//
// An unsigned code 0..15 in a byte is the E4M3 number code * 2^-9 (the
// subnormals and the first binade are one linear scale), so four codes of a
// word become an operand register by one AND.  x is scaled, group by group, by
// a power of two (the group's largest element to [2^7, 2^8)) and split, when
// the block starts, into three E4M3 parts of four bits each,
// x = p0 + p1 / 16 + p2 / 256: exact for elements down to 2^-14 (FP16) or
// 2^-17 (BF16) of the group's largest, and off by at most 2^-18 where the
// largest is 2^7, that is 2^-25 of it, below that -- less than the half step of
// 2^-24 by which an FP32 sum of the group with that element in it is rounded.  (Relative to the whole
// row's largest, an outlier would cost other groups their bits, also for the
// weight rows whose code at the outlier is the zero point.)  An infinity or a
// NaN makes its group's factor NaN, and so every output.  The parts are columns of
// the N side, and the products are added in FP32 by mma.m16n8k32 (checked:
// 24-bit sums, no shorter accumulator).
// Taken from two row tiles per block slot on: 28672 x 8192 in 34.7 us against
// 43.9 with 16-bit products, 14336 x 4096 in 13.0 against 14.7; below that the
// splitting of x costs more (4864 x 1024, 5 rows: 7.7 against 4.5), and more
// rows fill more columns with parts (14336 x 4096, 4 rows: 18.5 against 14.7).
// One block per SM from K of about 15400 on still wins while the parts fit 64
// KB (20000 x 16384: 60.5 us against 64.5, x 20480: 75.2 against 79.7).
template <int MT, int GB, bool BF>
__global__ void __launch_bounds__(MV_WARPS * 32, 2) matvec4_one_kernel(const __grid_constant__ Matvec4Args a, int tiles, int steps, int kw_log) {
    constexpr int NST = MV_ONE_STAGES;
    constexpr int STAGE = MT * 16 * MV_ROW;
    constexpr int NGS = 8 / GB;              // groups of a step
    constexpr int PARTS = MV_PARTS;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_index();
    const int g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * NST * STAGE;
    float* sm_sum = reinterpret_cast<float*>(smem + MV_WARPS * NST * STAGE);  // [warps][MT][16][2]
    uint8_t* sm_x = reinterpret_cast<uint8_t*>(sm_sum + MV_WARPS * MT * 32);  // [K / 32][PARTS][4][8]
    float* sm_unit = reinterpret_cast<float*>(sm_x + a.K * PARTS);            // [per_warp * warps][NGS] what a group's parts count
    after_previous();
    const int kg = a.K / a.group;
    // 2^kw_log warps share K (step = i * that + kw), the others take further rows
    const int kws = 1 << kw_log, kw = warp & (kws - 1), rw = warp >> kw_log;
    const int tile_rows = (MV_WARPS >> kw_log) * (MT * 16);
    const int per_warp = (steps + kws - 1) >> kw_log;  // steps of a warp and tile
    const int my_tiles = ((int)blockIdx.x < tiles) ? (tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    // Nothing below branches per lane, because the matrix instructions need
    // the whole warp together: weight rows beyond N read the last row again
    // (not stored), columns beyond K the last ones (their scale is zero).
    // The pipeline runs over (tile, step) pairs, issue side and use side.
    const int64_t row_bytes = a.K / 2;
    const int last_kb = a.K / 2 - 16;
    int is_tile = 0, is_step = 0, is_stage = 0;
    auto issue = [&]() {
        if (is_tile < my_tiles) {
            const int64_t row0 = (int64_t)(blockIdx.x + (int64_t)is_tile * gridDim.x) * tile_rows + rw * (MT * 16);
            const int r = lane >> 3;
            const int kb = min((is_step * kws + kw) * MV_ROW + (lane & 7) * 16, last_kb);
            uint8_t* s = ring + is_stage * STAGE + r * MV_ROW;
            const int sw0 = ((lane & 7) ^ r) << 4, sw1 = sw0 ^ 64;  // row & 7 is r or r + 4
            if (row0 + MT * 16 <= a.N) {
                const uint8_t* p = a.codes + (row0 + r) * row_bytes + kb;
#pragma unroll
                for (int i = 0; i < MT * 4; ++i, p += 4 * row_bytes)
                    cp_async_16_zfill(s + i * 4 * MV_ROW + (i & 1 ? sw1 : sw0), p, 16);
            } else {
#pragma unroll
                for (int i = 0; i < MT * 4; ++i)
                    cp_async_16_zfill(s + i * 4 * MV_ROW + (i & 1 ? sw1 : sw0),
                                      a.codes + min(row0 + r + i * 4, (int64_t)a.N - 1) * row_bytes + kb, 16);
            }
            if (++is_step == per_warp) {
                is_step = 0;
                ++is_tile;
            }
            if (++is_stage == NST) is_stage = 0;
        }
        cp_async_commit();
    };
    // Scales (in pairs) and zeros (in fours) of a step's groups for one row per
    // lane (MT = 1: twice), loaded a step ahead and not touched until then.
    uint32_t sc[(NGS + 1) / 2], zb[(NGS + 3) / 4];
    int sz_tile = 0, sz_step = 0;
    const bool whole_groups = kg % NGS == 0 && a.scales_aligned;
    auto fetch_sz = [&]() {
        const int64_t row = min((int64_t)(blockIdx.x + (int64_t)sz_tile * gridDim.x) * tile_rows + rw * (MT * 16) + (lane & (MT * 16 - 1)),
                                (int64_t)a.N - 1);
        const int gi0 = (sz_step * kws + kw) * NGS;
        if (whole_groups && gi0 < kg) {
            const int64_t at = row * kg + gi0;
            const uint16_t* sp = static_cast<const uint16_t*>(a.scales) + at;
            if constexpr (NGS == 8) {
                const uint4 v = *reinterpret_cast<const uint4*>(sp);
                sc[0] = v.x, sc[1] = v.y, sc[2] = v.z, sc[3] = v.w;
                const uint2 z = a.zeros ? *reinterpret_cast<const uint2*>(a.zeros + at) : make_uint2(0x08080808u, 0x08080808u);
                zb[0] = z.x, zb[1] = z.y;
            } else if constexpr (NGS == 4) {
                const uint2 v = *reinterpret_cast<const uint2*>(sp);
                sc[0] = v.x, sc[1] = v.y;
                zb[0] = a.zeros ? *reinterpret_cast<const uint32_t*>(a.zeros + at) : 0x08080808u;
            } else {
                sc[0] = *reinterpret_cast<const uint32_t*>(sp);
                zb[0] = a.zeros ? *reinterpret_cast<const uint16_t*>(a.zeros + at) : 0x0808u;
            }
        } else {  // one by one; groups beyond K get scale 0
#pragma unroll
            for (int i = 0; i < (NGS + 3) / 4; ++i) zb[i] = 0;
#pragma unroll
            for (int i = 0; i < NGS; ++i) {
                const int gi = min(gi0 + i, kg - 1);
                uint32_t v = static_cast<const uint16_t*>(a.scales)[row * kg + gi];
                v = gi0 + i < kg ? v : 0u;
                sc[i / 2] = i % 2 ? sc[i / 2] | v << 16 : v;
                zb[i / 4] |= (a.zeros ? (uint32_t)a.zeros[row * kg + gi] : 8u) << (8 * (i % 4));
            }
        }
        if (++sz_step == per_warp) {
            sz_step = 0;
            ++sz_tile;
        }
    };
#pragma unroll 1
    for (int i = 0; i < NST - 1; ++i) issue();
    fetch_sz();

    // x in parts, while the first codes are on their way: the k of a word's
    // low nibbles (0, 2, 4, 6), then of its high nibbles.  A group's vectors
    // lie in 4 * GB neighbouring lanes; those beyond K are whole groups, which
    // work on the last vector and store nothing.
    const int vecs = a.K / 8;
    for (int i0 = 0; i0 < vecs; i0 += MV_WARPS * 32) {
        const int i = i0 + tid;
        float f[8];
        x_floats<BF>(ld_128(static_cast<const uint16_t*>(a.x) + min(i, vecs - 1) * 8), f);
        uint32_t most = 0;  // (the bits of non-negative floats compare as they do, NaN above all)
#pragma unroll
        for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(f[j]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < 4 * GB; o <<= 1) most = max(most, __shfl_xor_sync(FULL_MASK, most, o));
        const int exponent = x_exponent(most);
        const float fwd = __uint_as_float((uint32_t)(127 + 7 - exponent) << 23);
        if (i < vecs) {
            if (i % (4 * GB) == 0)
                sm_unit[i / (4 * GB)] = __uint_as_float(most >= 0x7f800000u ? 0x7fc00000u : (uint32_t)(127 - 7 + exponent) << 23);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= fwd;
            uint8_t* to = sm_x + ((i >> 2) * PARTS * 4 + (i & 3)) * 8;
#pragma unroll
            for (int p = 0; p < PARTS; ++p, to += 32) {
                const uint32_t lo = e4m3_four(f[0], f[2], f[4], f[6]), hi = e4m3_four(f[1], f[3], f[5], f[7]);
                *reinterpret_cast<uint2*>(to) = make_uint2(lo, hi);
                if (p + 1 < PARTS) {  // what is left, times 16 (exact)
                    float2 u, v;
                    e4m3x4_to_float(lo, u, v);
                    f[0] = (f[0] - u.x) * 16.f, f[2] = (f[2] - u.y) * 16.f, f[4] = (f[4] - v.x) * 16.f, f[6] = (f[6] - v.y) * 16.f;
                    e4m3x4_to_float(hi, u, v);
                    f[1] = (f[1] - u.x) * 16.f, f[3] = (f[3] - u.y) * 16.f, f[5] = (f[5] - v.x) * 16.f, f[7] = (f[7] - v.y) * 16.f;
                }
            }
        }
    }
    for (int i = kg + tid; i < (per_warp << kw_log) * NGS; i += MV_WARPS * 32) sm_unit[i] = 0.f;  // beyond K
    __syncthreads();
    // The lane's column (the last part again beyond the parts: not stored), and
    // what a lane's two columns count: parts 0 and 1 (t = 0), part 2 (t = 1).
    const uint8_t* const x_col = sm_x + min(g, PARTS - 1) * 32 + t * 8;
    const float c_first = t == 0 ? 1.f : 1.f / 256, c_second = t == 0 ? 1.f / 16 : 0.f;
    const int last_blk = a.K / 32 - 1;

    int use_stage = 0;
    for (int tile = 0; tile < my_tiles; ++tile) {
        const int64_t row0 = (int64_t)(blockIdx.x + (int64_t)tile * gridDim.x) * tile_rows;
        float tot[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 2; ++j) tot[mt][j] = 0.f;

#pragma unroll 1
        for (int si = 0; si < per_warp; ++si) {
            const int step = si * kws + kw;
            uint32_t sz[NGS];  // scale | FP16 of zero << 16
            // 1024 + z by its bits, less 1024: z, exact
#pragma unroll
            for (int i = 0; i < NGS / 2; ++i) {
                const uint32_t zp = __byte_perm(zb[i / 2], 0u, i % 2 ? 0x4342 : 0x4140) | 0x64006400u;
                uint32_t zz;
                asm("sub.f16x2 %0, %1, %2;" : "=r"(zz) : "r"(zp), "r"(0x64006400u));
                sz[2 * i] = __byte_perm(sc[i], zz, 0x5410);
                sz[2 * i + 1] = __byte_perm(sc[i], zz, 0x7632);
            }
            cp_async_wait<NST - 2>();
            __syncwarp();
            issue();
            fetch_sz();
            const uint8_t* s = ring + use_stage * STAGE;
            if (++use_stage == NST) use_stage = 0;
#pragma unroll
            for (int grp = 0; grp < NGS; ++grp) {
                float acc[MT][4], xs[4];
#pragma unroll
                for (int bb = 0; bb < GB; ++bb) {
                    const int blk = grp * GB + bb;
                    const uint2 xb = *reinterpret_cast<const uint2*>(x_col + min(step * 8 + blk, last_blk) * (PARTS * 32));
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const int sw = ((blk ^ g) << 4) + 4 * t;
                        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(s + (mt * 16 + g) * MV_ROW + sw);
                        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(s + (mt * 16 + g + 8) * MV_ROW + sw);
                        const uint32_t w[4] = {w0 & 0x0f0f0f0fu, w1 & 0x0f0f0f0fu, w0 >> 4 & 0x0f0f0f0fu,
                                               w1 >> 4 & 0x0f0f0f0fu};
                        e4m3_mma(acc[mt], w, xb, bb == 0);
                    }
                    const uint32_t ones[4] = {0x38383838u, 0x38383838u, 0x38383838u, 0x38383838u};
                    e4m3_mma(xs, ones, xb, bb == 0);
                }
                // the parts together, all in units of 2^-9
                const float unit = sm_unit[step * NGS + grp];
                const float u_first = c_first * unit, u_second = c_second * unit;
                const float xsum = fmaf(xs[1], u_second, xs[0] * u_first) * (1.f / 512);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t v = __shfl_sync(FULL_MASK, sz[grp], mt * 16 + h * 8 + g);
                        float sc;
                        if (BF) {
                            sc = __uint_as_float(v << 16);
                        } else {
                            __half hh;
                            const uint16_t q = (uint16_t)v;
                            memcpy(&hh, &q, 2);
                            sc = __half2float(hh);
                        }
                        const float zz = __half2float(__ushort_as_half((uint16_t)(v >> 16)));
                        tot[mt][h] += sc * fmaf(-zz, xsum, fmaf(acc[mt][2 * h + 1], u_second, acc[mt][2 * h] * u_first));
                    }
            }
        }

        // the warps' sums, in their order
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (t < PARTS - 1) sm_sum[((warp * MT + mt) * 16 + h * 8 + g) * 2 + t] = tot[mt][h];
        __syncthreads();
        for (int r = tid; r < tile_rows; r += MV_WARPS * 32) {
            const int g0 = r / (MT * 16);
            const float* first = sm_sum + ((g0 << kw_log) * MT * 16 + r - g0 * (MT * 16)) * 2;
            float v = 0.f;
            for (int w = 0; w < kws; ++w) {
                v += first[w * MT * 32];
                v += first[w * MT * 32 + 1];
            }
            v *= 512.f;  // codes in units of 2^-9
            if (row0 + r < a.N) {
                if (BF)
                    static_cast<__nv_bfloat16*>(a.y)[row0 + r] = __float2bfloat16_rn(v);
                else
                    static_cast<__half*>(a.y)[row0 + r] = __float2half_rn(v);
            }
        }
        __syncthreads();
    }
    cp_async_wait<0>();
}

// Warps that share K, as a power of two: as many as there are steps, up to
// eight, so that none is idle on short rows (28672 x 512: 13.7 -> 4.8 us); four
// where eight would be idle for an eighth of their steps or more and half the
// blocks still fill the SMs (14336 x 2304, 8 rows: 17.7 -> 12.4 us; but 1152 x
// 4736 5.3 -> 7.4).
static int mv_kw_log(const Matvec4Args& a, const DeviceInfo& di) {
    const int steps = (a.K + MV_STEP - 1) / MV_STEP;
    if (steps < 8) return steps >= 4 ? 2 : steps >= 2 ? 1 : 0;
    const int by_eight = (steps + 7) / 8 * 8, by_four = (steps + 3) / 4 * 4;
    return by_four <= by_eight / 8 * 7 && a.N >= 32 * di.sm_count ? 2 : 3;
}
// Tiles of a block with two row tiles a warp.
static int mv_tiles2(const Matvec4Args& a, const DeviceInfo& di) {
    const int rows = (MV_WARPS >> mv_kw_log(a, di)) * 32;
    return (a.N - 1) / rows + 1;
}

// Enough weight rows to repay the splitting of x, whose parts fit shared
// memory beside the ring.
static bool one_row(const Matvec4Args& a, const DeviceInfo& di) {
    return a.T == 1 && mv_tiles2(a, di) >= 2 * di.sm_count && a.K * (int64_t)MV_PARTS <= 65536;
}

// A factor for each group of the steps that the warps take, those beyond K too.
static size_t mv_unit_bytes(const Matvec4Args& a, const DeviceInfo& di) {
    const int steps = (a.K + MV_STEP - 1) / MV_STEP, kws = 1 << mv_kw_log(a, di);
    return (size_t)(steps + kws - 1) / kws * kws * (MV_STEP / a.group) * 4;
}

template <int MT, int GB, bool BF>
static cudaError_t launch_mv_one(const Matvec4Args& a, const DeviceInfo& di, cudaStream_t st) {
    constexpr size_t fixed = (size_t)MV_WARPS * MV_ONE_STAGES * MT * 16 * MV_ROW + (size_t)MV_WARPS * MT * 32 * 4;
    const size_t smem = fixed + (size_t)a.K * MV_PARTS + mv_unit_bytes(a, di);
    auto kernel = matvec4_one_kernel<MT, GB, BF>;
    static SmemOnce once;
    const cudaError_t e = once.set(reinterpret_cast<const void*>(kernel), (int)fixed + 65536 + (65536 / MV_PARTS / MV_STEP + 8) * (MV_STEP / 32) * 4);
    if (e != cudaSuccess) return e;
    const int steps = (a.K + MV_STEP - 1) / MV_STEP, kw_log = mv_kw_log(a, di);
    const int tile_rows = (MV_WARPS >> kw_log) * MT * 16;
    const int tiles = (a.N - 1) / tile_rows + 1;
    const int per_sm = std::max(1, std::min(2, (int)((size_t)di.smem_per_sm / (smem + 1024))));
    return launch_after(kernel, dim3(std::min(tiles, di.sm_count * per_sm)), MV_WARPS * 32, smem, st, a, tiles, steps, kw_log);
}

template <int MT, bool BF>
static cudaError_t launch_mv_one_group(const Matvec4Args& a, const DeviceInfo& di, cudaStream_t st) {
    if (a.group == 32) return launch_mv_one<MT, 1, BF>(a, di, st);
    if (a.group == 64) return launch_mv_one<MT, 2, BF>(a, di, st);
    return launch_mv_one<MT, 4, BF>(a, di, st);
}

template <int MT, int NT, int GB, bool BF>
static cudaError_t launch_mv(const Matvec4Args& a, const DeviceInfo& di, cudaStream_t st) {
    constexpr int NST = mv_stages(MT);
    constexpr size_t smem = (size_t)MV_WARPS * NST * MT * 16 * MV_ROW + (size_t)MV_WARPS * MT * NT * 4 * 32 * 4;
    auto kernel = matvec4_kernel<MT, NT, GB, BF>;
    static SmemOnce once;
    cudaError_t e = once.set(reinterpret_cast<const void*>(kernel), (int)smem);
    if (e != cudaSuccess) return e;
    const int steps = (a.K + MV_STEP - 1) / MV_STEP, kw_log = mv_kw_log(a, di);
    const int tile_rows = (MV_WARPS >> kw_log) * MT * 16;
    const int tiles = (a.N - 1) / tile_rows + 1;
    const int per_sm = std::max(1, std::min(3, (int)((size_t)di.smem_per_sm / (smem + 1024))));
    const dim3 grid(std::min(tiles, di.sm_count * per_sm), (a.T + NT * 8 - 1) / (NT * 8));
    return launch_after(kernel, grid, MV_WARPS * 32, smem, st, a, tiles, steps, kw_log);
}

template <int MT, int NT, bool BF>
static cudaError_t launch_mv_group(const Matvec4Args& a, const DeviceInfo& di, cudaStream_t st) {
    if (a.group == 32) return launch_mv<MT, NT, 1, BF>(a, di, st);
    if (a.group == 64) return launch_mv<MT, NT, 2, BF>(a, di, st);
    return launch_mv<MT, NT, 4, BF>(a, di, st);
}

template <bool BF>
static cudaError_t launch_mv_rows(const Matvec4Args& a, const DeviceInfo& di, cudaStream_t st) {
    const bool two = mv_tiles2(a, di) >= di.sm_count;  // two row tiles a warp once they fill the SMs
    if (one_row(a, di)) return launch_mv_one_group<2, BF>(a, di, st);
    if (a.T <= 8) return two ? launch_mv_group<2, 1, BF>(a, di, st) : launch_mv_group<1, 1, BF>(a, di, st);
    if (a.T <= 16) return two ? launch_mv_group<2, 2, BF>(a, di, st) : launch_mv_group<1, 2, BF>(a, di, st);
    return two ? launch_mv_group<2, 4, BF>(a, di, st) : launch_mv_group<1, 4, BF>(a, di, st);
}

cudaError_t launch_matvec4(Matvec4Args a, int dtype, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    a.scales_aligned = reinterpret_cast<uintptr_t>(a.scales) % 16 == 0 && reinterpret_cast<uintptr_t>(a.zeros) % 8 == 0;
    return dtype == MOE_BF16 ? launch_mv_rows<true>(a, di, st) : launch_mv_rows<false>(a, di, st);
}

}  // namespace moedec
