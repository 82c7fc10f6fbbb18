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
// FP32's bits; the weights themselves are never rounded.
//
// Bound: HBM on the codes for few rows of x (half a byte per weight; scales
// and zero points add 3 bytes per group), then instruction issue: about ten
// instructions per eight codes and thread.  A warp takes 16 * MT weight rows
// (M of mma.m16n8k16) by 256 k per step through its own cp.async ring, eight
// rows of x are the N side, and the eight warps of a block split K, so a
// single token still has every warp of the GPU loading; their sums meet in
// shared memory once per tile, and blocks stride over the tiles with the ring
// running on across them.
#include <algorithm>

#include "common.cuh"
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

// Codes I and I + 4 of a word as the pair 16 + c (I = 0..3): the nibbles of
// the two 16-bit halves moved to the mantissa's top four bits.
template <bool BF, int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    constexpr int TOP = BF ? 3 : 6;  // lowest of the mantissa's top four bits
    constexpr int SH = 4 * I - TOP;
    const uint32_t v = SH >= 0 ? w >> (SH >= 0 ? SH : 0) : w << (SH < 0 ? -SH : 0);
    return (v & (0x000f000fu << TOP)) | (BF ? 0x41804180u : 0x4c004c00u);
}

}  // namespace

// GB: blocks of 32 k per group (1, 2, 4).
template <int MT, int NT, int GB, bool BF>
__global__ void __launch_bounds__(MV_WARPS * 32, NT <= 2 ? 2 : 1) matvec4_kernel(const __grid_constant__ Matvec4Args a, int tiles, int steps) {
    constexpr int NST = MT == 1 ? 4 : 3;
    constexpr int STAGE = MT * 16 * MV_ROW;
    constexpr int NGS = 8 / GB;              // groups of a step
    constexpr int SLOTS = (NGS + 3) / 4;     // of them in one lane
    constexpr int OUT = MT * NT * 4;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_index();
    const int g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * NST * STAGE;
    float* sm_sum = reinterpret_cast<float*>(smem + MV_WARPS * NST * STAGE);  // [warps][OUT][32]
    const int tok0 = blockIdx.y * (NT * 8);
    const int toks = min(a.T - tok0, NT * 8);
    const int kg = a.K / a.group;
    const int per_warp = (steps + MV_WARPS - 1) / MV_WARPS;  // steps of a warp and tile
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
            const int64_t row0 = (int64_t)(blockIdx.x + (int64_t)is_tile * gridDim.x) * (MT * 16);
            const int r = lane >> 3;
            const int kb = min((is_step * MV_WARPS + warp) * MV_ROW + (lane & 7) * 16, last_kb);
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
    // The lane's groups' scale | FP16 of 16 + zero << 16, one step ahead.
    uint32_t next_sz[MT][2][SLOTS];
    int sz_tile = 0, sz_step = 0;
    auto fetch_sz = [&]() {
        const int64_t row0 = (int64_t)(blockIdx.x + (int64_t)sz_tile * gridDim.x) * (MT * 16) + g;
        const int gi0 = (sz_step * MV_WARPS + warp) * NGS + (SLOTS == 1 && NGS < 4 ? t & (NGS - 1) : t);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int gi = min(gi0 + s * 4, kg - 1);
            const uint32_t keep = gi0 + s * 4 < kg ? 0xffffffffu : 0xffff0000u;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t at = min(row0 + mt * 16 + h * 8, (int64_t)a.N - 1) * kg + gi;
                    const uint32_t z = a.zeros ? __ldg(a.zeros + at) : 8u;
                    const uint32_t zz = __half_as_ushort(__uint2half_rn(16u + z));
                    next_sz[mt][h][s] = (__ldg(static_cast<const uint16_t*>(a.scales) + at) | zz << 16) & keep;
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
        const int64_t row0 = (int64_t)(blockIdx.x + (int64_t)tile * gridDim.x) * (MT * 16);
        float tot[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) tot[mt][nt][j] = 0.f;

#pragma unroll 1
        for (int si = 0; si < per_warp; ++si) {
            const int step = si * MV_WARPS + warp;
            uint32_t sz[MT][2][SLOTS];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int s = 0; s < SLOTS; ++s) sz[mt][h][s] = next_sz[mt][h][s];
            // x of the step first (L1 or L2), under the wait for the codes
            constexpr bool AHEAD = NT == 1;
            uint4 xv[AHEAD ? 8 : 1];
            if (AHEAD)
#pragma unroll
                for (int blk = 0; blk < 8; ++blk)
                    xv[blk % (AHEAD ? 8 : 1)] = ld_cached_128(xrow[0] + min(step * MV_STEP + blk * 32 + 8 * t, a.K - 8));
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
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        xs[nt][j] = 0.f;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) acc[mt][nt][j] = 0.f;
                    }
#pragma unroll
                for (int bb = 0; bb < GB; ++bb) {
                    const int blk = grp * GB + bb;
                    uint32_t xb[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 v = AHEAD ? xv[blk % (AHEAD ? 8 : 1)]
                                              : ld_cached_128(xrow[nt] + min(step * MV_STEP + blk * 32 + 8 * t, a.K - 8));
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
                            mv_mma<BF>(acc[mt][nt], a0, xb[nt][0], xb[nt][1]);
                            mv_mma<BF>(acc[mt][nt], a1, xb[nt][2], xb[nt][3]);
                        }
                    }
                    constexpr uint32_t one = BF ? 0x3f803f80u : 0x3c003c00u;
                    const uint32_t ones[4] = {one, one, one, one};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mv_mma<BF>(xs[nt], ones, xb[nt][0], xb[nt][1]);
                        mv_mma<BF>(xs[nt], ones, xb[nt][2], xb[nt][3]);
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t v = __shfl_sync(FULL_MASK, sz[mt][h][grp >> 2], (lane & 28) | (grp & 3));
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
        for (int e = tid; e < MT * 16 * toks; e += MV_WARPS * 32) {
            const int r = e % (MT * 16), tk = e / (MT * 16);
            const int mt = r >> 4, rg = r & 7, h = (r >> 3) & 1;
            const int nt = tk >> 3, tt = (tk & 7) >> 1, c = tk & 1;
            const int at = ((mt * NT + nt) * 4 + 2 * h + c) * 32 + rg * 4 + tt;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < MV_WARPS; ++w) v += sm_sum[w * OUT * 32 + at];
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

template <int MT, int NT, int GB, bool BF>
static cudaError_t launch_mv(const Matvec4Args& a, const DeviceInfo& di, cudaStream_t st) {
    constexpr int NST = MT == 1 ? 4 : 3;
    constexpr size_t smem = (size_t)MV_WARPS * NST * MT * 16 * MV_ROW + (size_t)MV_WARPS * MT * NT * 4 * 32 * 4;
    auto kernel = matvec4_kernel<MT, NT, GB, BF>;
    static SmemOnce once;
    cudaError_t e = once.set(reinterpret_cast<const void*>(kernel), (int)smem);
    if (e != cudaSuccess) return e;
    const int tiles = (a.N + MT * 16 - 1) / (MT * 16);
    const int steps = (a.K + MV_STEP - 1) / MV_STEP;
    const int per_sm = std::max(1, std::min(3, (int)((size_t)di.smem_per_sm / (smem + 1024))));
    const dim3 grid(std::min(tiles, di.sm_count * per_sm), (a.T + NT * 8 - 1) / (NT * 8));
    kernel<<<grid, MV_WARPS * 32, smem, st>>>(a, tiles, steps);
    return cudaGetLastError();
}

template <int MT, int NT, bool BF>
static cudaError_t launch_mv_group(const Matvec4Args& a, const DeviceInfo& di, cudaStream_t st) {
    if (a.group == 32) return launch_mv<MT, NT, 1, BF>(a, di, st);
    if (a.group == 64) return launch_mv<MT, NT, 2, BF>(a, di, st);
    return launch_mv<MT, NT, 4, BF>(a, di, st);
}

template <bool BF>
static cudaError_t launch_mv_rows(const Matvec4Args& a, const DeviceInfo& di, cudaStream_t st) {
    const bool two = (a.N + 31) / 32 >= di.sm_count;
    if (a.T <= 8) return two ? launch_mv_group<2, 1, BF>(a, di, st) : launch_mv_group<1, 1, BF>(a, di, st);
    if (a.T <= 16) return two ? launch_mv_group<2, 2, BF>(a, di, st) : launch_mv_group<1, 2, BF>(a, di, st);
    return two ? launch_mv_group<2, 4, BF>(a, di, st) : launch_mv_group<1, 4, BF>(a, di, st);
}

cudaError_t launch_matvec4(const Matvec4Args& a, int dtype, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    return dtype == MOE_BF16 ? launch_mv_rows<true>(a, di, st) : launch_mv_rows<false>(a, di, st);
}

}  // namespace moedec
