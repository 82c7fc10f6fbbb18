// internal.h -- launch interfaces between the C-ABI layer and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

namespace moedec {

struct MXView {
    const uint8_t* w;
    const uint8_t* s;
};

struct DecodeShape {
    int B, k, E, d, I, S;  // S = 1 with a shared expert
};

// Device properties cached per device (SM count, shared memory per block).
struct DeviceInfo {
    int sm_count;
    int max_smem_optin;
    int smem_per_sm;
    int* err_word;  // sticky device error bits (MOE_DEVERR_*)
};
cudaError_t device_info(DeviceInfo* out);

// h32: the intermediate is FP32 in the row-tile down pass's order (h32_pos)
// instead of the interface's BF16 [B][k+S][I]; the layer uses it when
// down_reads_h32() holds for its shape and weights.
cudaError_t launch_gate_up(const DecodeShape& s, const void* x, const int32_t* ids, MXView wg,
                           MXView wu, MXView shg, MXView shu, void* h, bool h32, cudaStream_t st);
cudaError_t launch_down(const DecodeShape& s, const void* h, bool h32, const int32_t* ids, const float* w,
                        MXView wd, MXView shd, void* y, cudaStream_t st, bool after_gate_up);
bool down_reads_h32(const DecodeShape& s, MXView wd, MXView shd);
cudaError_t launch_router(const float* logits, int B, int E, int k, int score, float scale, int32_t* ids, float* w,
                          cudaStream_t st);
cudaError_t launch_mx_requant(const void* in, void* out, int64_t rows, int K, cudaStream_t st);
cudaError_t launch_gate_up_fp4(const DecodeShape& s, const void* x, const int32_t* ids, MXView wg, MXView wu,
                               MXView shg, MXView shu, void* h, cudaStream_t st);
// The grouped (one pass over each distinct expert's rows) kernels with MXFP4
// weights: return false, launching nothing, when the shape or alignment
// does not suit them; else launch and set *err.
bool launch_gate_up_grouped_fp4(const DecodeShape& s, const void* x, const int32_t* ids, MXView wg, MXView wu,
                                MXView shg, MXView shu, void* h, cudaStream_t st, cudaError_t* err);
bool launch_down_grouped_fp4(const DecodeShape& s, const void* h, const int32_t* ids, const float* w, MXView wd,
                             MXView shd, void* y, cudaStream_t st, cudaError_t* err);
cudaError_t launch_down_fp4(const DecodeShape& s, const void* h, const int32_t* ids, const float* w, MXView wd,
                            MXView shd, void* y, cudaStream_t st);
// Shared-memory bytes the decode kernels need; 0 if the shape is beyond the
// supported limits.
size_t gate_up_smem_bytes(const DecodeShape& s);
size_t down_smem_bytes(const DecodeShape& s);

cudaError_t launch_align(const int32_t* ids, int T, int k, int E, int block_size, int32_t* sorted,
                         int64_t n_sorted, int32_t* expert_ids, int64_t n_blocks, int32_t* ntpp,
                         void* ws, cudaStream_t st);
size_t align_workspace_bytes(int64_t n, int E);
size_t align_smem_bytes(int E);
// Device address of the library's fixed align scratch on the current device.
cudaError_t align_static_scratch(void** out);

cudaError_t launch_copy(void* dst, const void* src, size_t bytes, cudaStream_t st);

// The expert-centric (grouped GEMM) layer's device buffers, carved from the
// caller's workspace.
struct GroupedWorkspace {
    int32_t* sorted;      // [n_sorted] flat slot of each sorted row (T*k = pad)
    int64_t n_sorted;
    int32_t* expert_ids;  // [n_blocks]
    int64_t n_blocks;
    int32_t* ntpp;        // rows used, a multiple of the block size
    void* align_ws;
    uint16_t* x_mx;       // [T][d] x rounded through MXFP8 (act_mx only)
    uint16_t* h_sorted;   // [n_sorted][I] BF16
    float* out;           // [T*k][d] FP32 per-slot partial outputs
    // the shared expert's pass (null without one): every token, in order
    int32_t* sh_sorted;   // [n_sh] token of each row (T = pad)
    int32_t* sh_expert;   // [n_sh / 128] all 0
    int32_t* sh_ntpp;     // n_sh
    int64_t n_sh;         // T rounded up to a multiple of 128
    uint16_t* sh_h;       // [n_sh][I] BF16
    float* sh_out;        // [T][d] FP32
};
constexpr int GROUPED_BLOCK = 128;  // sorted rows per block
bool grouped_shape_ok(int d, int I);
size_t grouped_smem_bytes(int d, int I);
// shg / shu / shd: the shared expert's matrices ([1][rows][K]) or all null.
cudaError_t launch_grouped(const uint16_t* x, int T, int d, const int32_t* ids, const float* w, int k, MXView wg,
                           MXView wu, MXView wd, MXView shg, MXView shu, MXView shd, int E, int I, bool act_mx,
                           const GroupedWorkspace& ws, uint16_t* y, cudaStream_t st);

// Raises a kernel's dynamic shared memory limit once per device.
struct SmemOnce {
    std::mutex mu;
    bool have[64] = {false};
    cudaError_t set(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lock(mu);
        if (have[dev]) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) have[dev] = true;
        return e;
    }
};

// Paged attention: blocks of a launch at most (a join counter and two pieces
// of workspace each), and the counters' bytes at the start of the workspace.
constexpr int ATTN_MAX_BLOCKS = 640;
constexpr size_t ATTN_COUNTER_BYTES = 4096;  // MOE_ATTN_COUNTER_BYTES
static_assert((ATTN_MAX_BLOCKS + 2 * (ATTN_MAX_BLOCKS / 8 + 1)) * 4 <= ATTN_COUNTER_BYTES, "a counter per block, two per eight");
struct AttnArgs {
    const void* q;
    int64_t q_sb, q_sh;  // strides in elements, here and below
    const void* k;
    int64_t k_sp, k_st, k_sh;  // page, token, head
    const void* v;
    int64_t v_sp, v_st, v_sh;
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lens;
    int B, Hq, Hkv, D, num_pages, page, max_pages, window, sinks;
    float scale_log2, v_scale;
    void* out;
    float* lse;
    // the part behind a shared prefix (part_o not null): sequences that share it
    // (shares null: all) and reach its end begin at token `first`, and (m, l) and
    // the unnormalised sums [B][Hq][D] go to part_ml, part_o in place of out
    int first;
    const uint8_t* shares;
    float* part_o;
    float* part_ml;
    // filled by the launch
    bool out_aligned;    // to 8 bytes
    uint32_t page_mul;
    int page_shift;
    int G, hpi, chunks;  // query heads of a key-value head, of an item; items of a group
    int* counters;
    float* ws_ml;  // [2 * blocks][hpi][2] maximum and sum of a piece
    float* ws_o;   // [2 * blocks][hpi][D]
    int* err;
};
size_t attn_workspace_bytes(int Hq, int Hkv, int D);
cudaError_t launch_paged_attention(AttnArgs a, int dtype, int cache_dtype, void* ws, cudaStream_t st);

// Attention of a batch with a shared prefix; `own` in launch_shared_prefix is
// the call on the sequences' own keys.
constexpr int PX_MAX_BLOCKS = 160;  // of a prefix launch that cuts the prefix (one per SM)
struct PrefixArgs {
    const void* q;
    int64_t q_sb, q_sh;  // strides in elements, here and below
    const void* k;
    int64_t k_sp, k_st, k_sh;  // page, token, head
    const void* v;
    int64_t v_sp, v_st, v_sh;
    const int32_t* table;  // pages of the prefix
    const int32_t* lens;
    const uint8_t* shares;
    int len;      // tokens of the prefix
    int64_t cap;  // tokens that a row of the block table holds
    int B, Hq, Hkv, D, num_pages, page;
    float scale_log2, v_scale;
    void* out;
    float* lse;
    // filled by the launch
    bool out_aligned;
    uint32_t page_mul;
    int page_shift;
    int G, group_rows, splits, pieces, join_groups;
    float* own_o;   // [B][Hq][D]
    float* own_ml;  // [B][Hq][2]
    float* ws_o;    // [Hkv][pieces][B * G][D]
    float* ws_ml;   // [Hkv][pieces][B * G][2]
    int* err;
};
size_t prefix_workspace_bytes(int B, int Hq, int Hkv, int D);
bool prefix_pays(int B, int Hkv, int D, int len, bool e4);
cudaError_t launch_shared_prefix(PrefixArgs a, const AttnArgs& own, int dtype, int cache_dtype, void* ws, cudaStream_t st);

struct RopeArgs {
    const void* q;
    int64_t q_st, q_sh;  // token, head
    const void* k;
    int64_t k_st, k_sh;
    const void* v;
    int64_t v_st, v_sh;
    void* q_out;
    int64_t qo_st, qo_sh;
    void* kc;
    int64_t kc_sp, kc_st, kc_sh;
    void* vc;
    int64_t vc_sp, vc_st, vc_sh;
    const int32_t* positions;
    const int64_t* slots;
    const double* freqs;
    int T, Hq, Hkv, D, rot, interleaved, num_pages, page;
    float mscale, k_scale, v_scale;
    float k_inv, v_inv;  // filled by the launch
    int* err;
};
cudaError_t launch_rope_append(RopeArgs a, int dtype, int cache_dtype, cudaStream_t st);

struct NormSpec {
    const void* w;
    const void* b;
    float eps;
    int kind;  // MOE_NORM_*; -1: no norm
};
struct NormArgs {
    const void* y;
    int64_t y_stride;
    const void* resid;
    int64_t r_stride;
    const void* gate;
    int64_t gate_row, gate_col;  // strides in elements (0 broadcasts)
    int gate_act;
    float alpha;
    NormSpec post, pre;
    void* resid_out;
    void* out;
    int T, d;
};
cudaError_t launch_norm_residual(const NormArgs& a, int dtype, int resid_dtype, cudaStream_t st);

struct Matvec4Args {
    const void* x;
    int64_t x_stride;
    const uint8_t* codes;
    const void* scales;
    const uint8_t* zeros;
    void* y;
    int64_t y_stride;
    int T, N, K, group;
    bool scales_aligned;  // filled by the launch
};
cudaError_t launch_matvec4(Matvec4Args a, int dtype, cudaStream_t st);

struct RouterGroupedArgs {
    const void* logits;
    int64_t stride;  // of a row, in elements
    const float* bias;
    int T, E, k, score, groups, top_groups, group_score, renorm;
    float scale;
    int32_t* ids;
    float* w;
    // filled by the launch
    bool vec;  // four logits at a time
    int* err;
};
cudaError_t launch_router_grouped(RouterGroupedArgs a, int dtype, cudaStream_t st);

constexpr int PAGES_MAX_BATCH = 4096;  // MOE_PAGES_MAX_BATCH
enum { PAGES_ROWS = 1, PAGES_STATE = 2 };
struct PagesArgs {
    const int32_t* past;    // lengths before
    const int32_t* news;    // plan: new tokens
    const uint8_t* ended;   // release
    const uint8_t* shares;  // or null: all
    const int32_t* shared;
    int shared_n;
    int32_t* table;
    int64_t table_stride;
    int32_t* free_pages;
    int capacity;
    const int32_t* n_free;
    int B, T, max_pages, page;
    int32_t* positions;
    int64_t* slots;
    int32_t* seq_ids;
    int32_t* starts;
    int32_t* lens_out;
    int32_t* n_free_out;
    // filled by the launch
    bool vec;   // outputs of tokens aligned to 16 bytes
    int parts;  // what a launch writes: PAGES_ROWS, PAGES_STATE
    int* err;
};
cudaError_t launch_plan_pages(PagesArgs a, cudaStream_t st);
cudaError_t launch_release_pages(PagesArgs a, cudaStream_t st);

}  // namespace moedec
