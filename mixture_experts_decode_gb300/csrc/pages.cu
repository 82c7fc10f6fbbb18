// pages.cu -- the bookkeeping of a paged cache on the device: from the
// requests' lengths, the pages that new tokens need (from a stack of free
// ones), block tables, positions, slots and the new lengths; and the pages of
// requests that have ended back onto the stack.
//
// Every block scans the batch (two sums per request) in shared memory, then
// takes its share of the tokens (or pages), each found by a binary search in
// the scan: nothing is handed from one block to another, so one launch does
// all of it.  Lengths and the stack's height may be updated in place; a call
// of several blocks then writes them in a launch of its own, which begins when
// all blocks have read them (it waits for what they still write at its end, so
// that what follows finds everything).  That launch reads before any wait of
// its own, so what it reads, the last call's results among it, is read past L1.
// Bound: latency for a decode step (64 requests: 5.1 us); for long prompts
// the 16 bytes written per token behind it (500 requests, 889 000 tokens: 10.9 us).
#include <algorithm>

#include "block_common.cuh"
#include "internal.h"

namespace moedec {

namespace {

constexpr int PG_THREADS = 512;
constexpr int PG_ITEMS = PAGES_MAX_BATCH / PG_THREADS;  // requests per thread
constexpr int PG_GROUP = 4;                             // tokens (or pages) per thread and pass

struct Pair {
    int64_t a, b;
};
__device__ __forceinline__ Pair operator+(Pair x, Pair y) { return {x.a + y.a, x.b + y.b}; }

// Exclusive sums over the block's threads of v, in order; *all gets the total.
__device__ __forceinline__ Pair block_exclusive(Pair v, Pair* all) {
    __shared__ Pair part[PG_THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto scan = [&](Pair s, int width) {  // inclusive, over `width` lanes
        for (int o = 1; o < width; o <<= 1) {
            const Pair u = {__shfl_up_sync(FULL_MASK, s.a, o), __shfl_up_sync(FULL_MASK, s.b, o)};
            if (lane >= o) s = s + u;
        }
        return s;
    };
    const Pair s = scan(v, 32);
    __syncthreads();  // (the last use of part is over)
    if (lane == 31) part[warp] = s;
    __syncthreads();
    // every warp scans the warps' sums for itself
    constexpr int WARPS = PG_THREADS / 32;
    const Pair t = scan(part[lane < WARPS ? lane : 0], WARPS);
    *all = {__shfl_sync(FULL_MASK, t.a, WARPS - 1), __shfl_sync(FULL_MASK, t.b, WARPS - 1)};
    Pair before = {__shfl_sync(FULL_MASK, t.a, warp > 0 ? warp - 1 : 0), __shfl_sync(FULL_MASK, t.b, warp > 0 ? warp - 1 : 0)};
    if (warp == 0) before = {0, 0};
    return {before.a + s.a - v.a, before.b + s.b - v.b};
}

// The last of begin[0 .. n) that is at most i (begin[0] = 0 <= i).
__device__ __forceinline__ int last_at_most(const int32_t* begin, int n, int i) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (begin[mid] <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// ceil(tokens / page), for all of 32 bits (64-bit quotients take several times as long).
__device__ __forceinline__ uint32_t pages_of(uint32_t tokens, uint32_t page) {
    const uint32_t q = tokens / page;
    return q + (q * page != tokens);
}

// What the calls before may have written.  The state's launch has not waited
// for anything itself: its loads go past L1, whose lines may be older.  (For all
// launches, 304 blocks then ask the L2 for the same lines: 1000 requests of which
// 900 end 5.9 us in place of 5.4.)
template <class T>
__device__ __forceinline__ T read(const PagesArgs& a, const T* p) {
    return a.parts == PAGES_STATE ? __ldcg(p) : *p;
}

__device__ __forceinline__ int stack_height(const PagesArgs& a) {
    const int n = read(a, a.n_free);
    if (blockIdx.x == 0 && threadIdx.x == 0 && (n < 0 || n > a.capacity)) atomicOr(a.err, MOE_DEVERR_POOL);
    return min(max(n, 0), a.capacity);
}

}  // namespace

// Tokens: request b's new ones are starts[b] .. starts[b + 1) of the outputs.
__global__ void __launch_bounds__(PG_THREADS) plan_pages_kernel(const __grid_constant__ PagesArgs a) {
    extern __shared__ int32_t sm[];
    int32_t* const starts = sm;             // [B + 1] first token
    int32_t* const past = starts + a.B + 1; // [B]
    int32_t* const base = past + a.B;       // [B] first new page, counted from the stack's top
    if (a.parts != PAGES_STATE) after_previous();
    const int tid = threadIdx.x;
    const int height = stack_height(a);
    const int64_t cap = min((int64_t)a.max_pages * a.page, (int64_t)INT32_MAX);

    // what each request asks for, and whether it fits behind those before it
    const int per = (a.B + PG_THREADS - 1) / PG_THREADS;
    int news[PG_ITEMS], needs[PG_ITEMS];
    Pair sum = {0, 0}, all;
    bool refused = false;
#pragma unroll
    for (int i = 0; i < PG_ITEMS; ++i) {
        const int b = tid * per + i;
        news[i] = needs[i] = 0;
        if (i < per && b < a.B) {
            const int p = read(a, a.past + b), n = read(a, a.news + b);
            past[b] = p;
            if (p < 0 || n < 0) {
                refused = true;
                news[i] = -1;
            } else {
                news[i] = n;
                needs[i] = (int)(pages_of((uint32_t)p + (uint32_t)n, a.page) - pages_of(p, a.page));  // at most n
                sum = sum + Pair{n, needs[i]};
            }
        }
    }
    const Pair first = block_exclusive(sum, &all);
    Pair at = first, got = {0, 0};
    bool dropped = false;
#pragma unroll
    for (int i = 0; i < PG_ITEMS; ++i) {
        const int b = tid * per + i;
        if (i < per && b < a.B) {
            if (news[i] < 0) {
                news[i] = 0;
                continue;
            }
            at = at + Pair{news[i], needs[i]};
            const bool fits = at.a <= a.T && (needs[i] == 0 || at.b <= height) && (int64_t)past[b] + news[i] <= cap;
            if (!fits) {
                dropped |= news[i] > 0;
                news[i] = needs[i] = 0;
            }
            got = got + Pair{news[i], needs[i]};
        }
    }
    at = first;
    if (__syncthreads_or(dropped)) {  // the sums of what is left
        refused |= dropped;
        at = block_exclusive(got, &all);
    }
#pragma unroll
    for (int i = 0; i < PG_ITEMS; ++i) {
        const int b = tid * per + i;
        if (i < per && b < a.B) {
            starts[b] = (int)at.a;
            base[b] = (int)at.b;
            at = at + Pair{news[i], needs[i]};
        }
    }
    if (tid == 0) starts[a.B] = (int)all.a;
    if (refused && blockIdx.x == 0) atomicOr(a.err, MOE_DEVERR_POOL);
    __syncthreads();
    const int total = starts[a.B];

    if (a.parts & PAGES_STATE) {
        if (blockIdx.x == 0) {
            for (int b = tid; b < a.B; b += PG_THREADS) a.lens_out[b] = past[b] + starts[b + 1] - starts[b];
            if (tid == 0) *a.n_free_out = height - (int)all.b;
        }
        if (!(a.parts & PAGES_ROWS)) {
            after_previous();
            return;
        }
    }
    if (a.parts == PAGES_ROWS) let_next_start();  // (all that the state's launch writes has been read)
    if (blockIdx.x == 0)
        for (int b = tid; b <= a.B; b += PG_THREADS) a.starts[b] = starts[b];
    // requests that begin behind the shared prefix: its pages
    if (a.shared_n > 0) {
        const int entries = min(a.shared_n, a.max_pages);
        const int warp = tid >> 5, lane = tid & 31;
        for (int b = blockIdx.x + gridDim.x * warp; b < a.B; b += gridDim.x * (PG_THREADS / 32))
            if (starts[b + 1] > starts[b] && past[b] == (int64_t)a.shared_n * a.page && (!a.shares || a.shares[b]))
                for (int i = lane; i < entries; i += 32) a.table[b * a.table_stride + i] = a.shared[i];
    }
    for (int64_t t0 = ((int64_t)blockIdx.x * PG_THREADS + tid) * PG_GROUP; t0 < a.T;
         t0 += (int64_t)gridDim.x * PG_THREADS * PG_GROUP) {
        const int n = (int)min((int64_t)PG_GROUP, a.T - t0);
        int32_t pos[PG_GROUP], seq[PG_GROUP];
        int64_t slot[PG_GROUP];
        int b = t0 < total ? last_at_most(starts, a.B, (int)t0) : a.B;
        int p = 0, pi = 0, off = 0, have = 0, pg = 0;
        bool found = false;  // p .. have are of request b
#pragma unroll
        for (int i = 0; i < PG_GROUP; ++i) {
            const int t = (int)t0 + i;
            pos[i] = 0, seq[i] = -1, slot[i] = -1;
            if (t0 + i < total) {
                while (starts[b + 1] <= t) ++b, found = false;
                if (!found) {
                    p = past[b] + (t - starts[b]);
                    pi = (int)((uint32_t)p / (uint32_t)a.page), off = p - pi * a.page;
                    have = (int)pages_of(past[b], a.page);
                } else if (++p, ++off == a.page) {
                    off = 0, ++pi;
                }
                if (!found || off == 0) {
                    int32_t* const entry = a.table + b * a.table_stride + pi;
                    if (pi < have) {
                        pg = *entry;
                    } else {
                        pg = a.free_pages[height - 1 - (base[b] + pi - have)];
                        if (off == 0) *entry = pg;  // the page's first token puts it into the table
                    }
                    if (pg < 0) atomicOr(a.err, MOE_DEVERR_PAGE);
                    found = true;
                }
                pos[i] = p, seq[i] = b;
                slot[i] = pg < 0 ? -1 : (int64_t)pg * a.page + off;
            }
        }
        if (n == PG_GROUP && a.vec) {
            *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4*>(a.seq_ids + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
            *reinterpret_cast<longlong2*>(a.slots + t0) = make_longlong2(slot[0], slot[1]);
            *reinterpret_cast<longlong2*>(a.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
        } else {
            for (int i = 0; i < n; ++i) {
                a.positions[t0 + i] = pos[i];
                a.seq_ids[t0 + i] = seq[i];
                a.slots[t0 + i] = slot[i];
            }
        }
    }
}

// Pages of ended requests, in the order of requests and of their pages.
__global__ void __launch_bounds__(PG_THREADS) release_pages_kernel(const __grid_constant__ PagesArgs a) {
    extern __shared__ int32_t sm[];
    int32_t* const begin = sm;            // [B + 1] first page among those that go
    int32_t* const after = begin + a.B + 1;  // [B] the lengths behind it
    int32_t* const skip = after + a.B;    // [B] pages that stay, the shared ones
    if (a.parts != PAGES_STATE) after_previous();
    const int tid = threadIdx.x;
    const int height = stack_height(a);
    const int per = (a.B + PG_THREADS - 1) / PG_THREADS;
    int goes[PG_ITEMS];
    Pair sum = {0, 0}, all;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PG_ITEMS; ++i) {
        const int b = tid * per + i;
        goes[i] = 0;
        if (i < per && b < a.B) {
            const int p = read(a, a.past + b);
            const bool ends = read(a, a.ended + b) != 0;
            skip[b] = !a.shares || read(a, a.shares + b) ? a.shared_n : 0;
            after[b] = ends ? 0 : p;
            if (ends) {
                const int64_t have = p < 0 ? 0 : pages_of(p, a.page);
                if (p < 0 || have > a.max_pages) bad = true;
                goes[i] = max(0, (int)min(have, (int64_t)a.max_pages) - skip[b]);
                sum.a += goes[i];
            }
        }
    }
    Pair at = block_exclusive(sum, &all);
    const int room = a.capacity - height;
    if (all.a > room) bad = true;
    if (bad && blockIdx.x == 0) atomicOr(a.err, MOE_DEVERR_POOL);
    const int total = (int)min(all.a, (int64_t)room);
#pragma unroll
    for (int i = 0; i < PG_ITEMS; ++i) {
        const int b = tid * per + i;
        if (i < per && b < a.B) {
            begin[b] = (int)min(at.a, (int64_t)total);
            at.a += goes[i];
        }
    }
    if (tid == 0) begin[a.B] = total;
    __syncthreads();
    if (a.parts & PAGES_STATE) {
        if (blockIdx.x == 0) {
            for (int b = tid; b < a.B; b += PG_THREADS) a.lens_out[b] = after[b];
            if (tid == 0) *a.n_free_out = height + total;
        }
        if (!(a.parts & PAGES_ROWS)) {
            after_previous();
            return;
        }
    }
    if (a.parts == PAGES_ROWS) let_next_start();  // (all that the state's launch writes has been read)
    for (int64_t i0 = ((int64_t)blockIdx.x * PG_THREADS + tid) * PG_GROUP; i0 < total;
         i0 += (int64_t)gridDim.x * PG_THREADS * PG_GROUP) {
        int b = last_at_most(begin, a.B, (int)i0);
#pragma unroll
        for (int j = 0; j < PG_GROUP; ++j) {
            const int i = (int)i0 + j;
            if (i >= total) break;
            while (begin[b + 1] <= i) ++b;
            const int pg = a.table[b * a.table_stride + skip[b] + (i - begin[b])];
            if (pg < 0) atomicOr(a.err, MOE_DEVERR_PAGE);
            a.free_pages[height + i] = pg;
        }
    }
}

static bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

static cudaError_t launch_pages(void (*kernel)(PagesArgs), SmemOnce& once, PagesArgs a, int64_t rows, size_t smem,
                                cudaStream_t st) {
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    e = once.set(reinterpret_cast<const void*>(kernel), 64 * 1024);
    if (e != cudaSuccess) return e;
    a.err = di.err_word;
    const int64_t tiles = std::max<int64_t>(1, (rows + PG_THREADS * PG_GROUP - 1) / (PG_THREADS * PG_GROUP));
    const int grid = (int)std::min<int64_t>(tiles, di.sm_count * 2);
    const size_t lens = (size_t)a.B * 4;
    const bool in_place = overlaps(a.past, lens, a.lens_out, lens) || overlaps(a.n_free, 4, a.n_free_out, 4) ||
                          (a.news && overlaps(a.news, lens, a.lens_out, lens));
    a.parts = PAGES_ROWS | PAGES_STATE;
    if (grid == 1 || !in_place) return launch_after(kernel, dim3(grid), PG_THREADS, smem, st, a);
    a.parts = PAGES_ROWS;
    e = launch_after(kernel, dim3(grid), PG_THREADS, smem, st, a);
    if (e != cudaSuccess) return e;
    a.parts = PAGES_STATE;
    return launch_after(kernel, dim3(1), PG_THREADS, smem, st, a);
}

cudaError_t launch_plan_pages(PagesArgs a, cudaStream_t st) {
    a.vec = reinterpret_cast<uintptr_t>(a.positions) % 16 == 0 && reinterpret_cast<uintptr_t>(a.seq_ids) % 16 == 0 &&
            reinterpret_cast<uintptr_t>(a.slots) % 16 == 0;
    static SmemOnce once;
    return launch_pages(plan_pages_kernel, once, a, a.T, ((size_t)a.B * 3 + 1) * 4, st);
}

cudaError_t launch_release_pages(PagesArgs a, cudaStream_t st) {
    static SmemOnce once;
    return launch_pages(release_pages_kernel, once, a, (int64_t)a.B * a.max_pages / 4, ((size_t)a.B * 3 + 1) * 4, st);
}

}  // namespace moedec
