// Internal interface between the C ABI (abi.cpp) and the kernel launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "nvfp4kv.h"

namespace nvfp4kv {

constexpr int kPageSize = 16;
constexpr int kHeadDim = 128;
constexpr int kMaxGroup = 8;                 // query heads per kv head handled by one warp
constexpr int kDecodeWarps = 16;             // warps (independent workers) per decode CTA
constexpr int kDecodeCtasPerSm = 1;          // occupancy the default worker count assumes
constexpr int kPartialFloats = kMaxGroup * kHeadDim + 2 * kMaxGroup;  // O[8][128], m[8], l[8]
constexpr int kNvfp4Record = 2304;           // bytes of an NVFP4 page-head record
constexpr int kFp8Record = 4096;             // bytes of an FP8 page-head record
constexpr int kFp8BlockRecord = FP8BKV_RECORD_BYTES;  // ... of one with its scales of K and V behind it
constexpr int kMaxBatch = NVFP4KV_MAX_BATCH; // prefix table lives in shared memory
constexpr int kMaxScaledHeads = NVFP4KV_MAX_SCALED_KV_HEADS;
// Polls before a wait for staged data (or for another role of the CTA) gives
// up and reports NVFP4KV_DEV_TIMEOUT; the launching calls pass the current
// process-wide limit (nvfp4kv_set_wait_limit) in the kernels' parameters.  A
// wait that only lets work already in flight land before the CTA exits always
// uses this default, whatever the setting.
constexpr uint32_t kWaitLimit = NVFP4KV_WAIT_LIMIT_DEFAULT;

// Per-kv-head tensor scales of K and V, fl32(G * factor), used when per_head
// is set (kernels take these parameters as __grid_constant__, so a head index
// reads them in place); otherwise every head uses the uniform scale.
struct HeadScales {
    int per_head;
    float k[kMaxScaledHeads];
    float v[kMaxScaledHeads];
};

// What a decode over few pages needs (launched by clusters, without partials); the
// per-head scales, two thirds of the full parameters, only where there are any.
struct ClusterParams {
    const uint8_t *pool;
    const uint16_t *q;
    void *out;
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *sel_pages;    // null: all pages
    int32_t *dev_status;
    int hq;
    int hkv;
    int group;
    int max_pages;
    int num_pages;
    int budget;
    int sel_q_len;
    int out_bf16;
    float qscale;
    float out_scale;
    uint32_t wait_limit;
    int seg0;                    // the launch's first (query token, kv head)
};

struct ClusterHeadParams : ClusterParams {
    float qs[kMaxScaledHeads];   // query scale and output scale of each kv head
    float vs[kMaxScaledHeads];
};

// Split-KV decode over either cache format.
struct DecodeParams {
    const uint8_t *pool;         // page-head records [num_pages][hkv][record]
    const uint16_t *q;           // bf16 [batch][hq][128]
    void *out;                   // [batch][hq][128] bf16 or f32
    const int32_t *block_table;  // [batch][max_pages]
    const int32_t *seq_lens;     // [batch]
    int32_t *dev_status;         // nullable
    float *partials;             // [2 * num_workers][kPartialFloats]
    int batch;
    int hq;
    int hkv;
    int group;
    int max_pages;
    int num_pages;
    int out_bf16;
    int num_workers;
    float qscale;                // sm_scale * log2(e) * tensor scale
    float out_scale;             // tensor scale of V (1 for the FP8 cache)
    float gscale;                // tensor scale the fused append divides by
    // fused append: new K/V rows [batch][hkv][128] written at position
    // seq_lens[b] - 1 before the decode reads the page (append != 0)
    const void *k_new;
    const void *v_new;
    int append;
    int new_bf16;
    // multi-query decode: q_len query tokens per sequence (the last q_len
    // positions, causal among themselves); rows = group * q_len query rows
    // per kv head, taken in row groups of kMaxGroup
    int q_len;
    int rows;
    int row_groups;
    int lanes;                   // row groups that neighbouring workers take side by side: row_groups, or 1
    // per-head tensor scales (NVFP4): append divisors and V output scales,
    // and the query scale sm_scale * log2(e) * G_k,h of each kv head
    HeadScales hs;
    float qs[kMaxScaledHeads];
    uint32_t wait_limit;         // polls before a wait gives up (kWaitLimit by default)
    // attention over listed pages: `batch` counts query tokens, sel_q_len of a
    // sequence; sel_pages [batch][hkv][budget] pages of the sequence
    const int32_t *sel_pages;
    int budget;
    int sel_q_len;
};

struct QuantParams {
    const void *k_new;
    const void *v_new;
    const int32_t *slot_mapping;
    uint8_t *pool;               // page-head records [num_pages][hkv][record]
    int32_t *dev_status;
    int num_tokens;
    int hkv;
    int num_pages;
    int in_bf16;
    float gscale;                // tensor scale: blocks are taken of x / gscale
    HeadScales hs;
};

struct PrefixParams {
    const uint8_t *pool;         // NVFP4 page-head records
    const int32_t *block_table;
    const int32_t *prefix_lens;
    const int32_t *kv_indptr;
    uint8_t *k_out;
    uint8_t *v_out;
    int32_t *dev_status;
    int batch;
    int hkv;
    int max_pages;
    int num_pages;
    float gscale;                // tensor scale multiplying every value
    HeadScales hs;
    uint32_t wait_limit;         // polls before a wait gives up (kWaitLimit by default)
};

struct ExtendParams {
    const uint16_t *q;           // bf16 [q rows][hq][128]
    const int32_t *q_indptr;     // [batch + 1] chunk row ranges
    const uint8_t *k_prefix;     // E4M3 [prefix rows][hkv][128]
    const uint8_t *v_prefix;
    const int32_t *kv_indptr;    // [batch] first prefix row of each sequence
    const int32_t *prefix_lens;  // [batch]
    const void *k_chunk;         // [q rows][hkv][128]: bf16, or E4M3 bytes when chunk_e4m3
    const void *v_chunk;
    void *out;                   // [q rows][hq][128], bf16 or fp32
    int32_t *dev_status;
    int batch;
    int hq;
    int hkv;
    int group;                   // hq / hkv
    int q_rows;                  // rows of q, k_chunk, v_chunk and out
    int max_q_len;               // bound on every chunk length (sizes the grid)
    int64_t prefix_rows;         // rows of the prefix workspace
    float qscale;                // sm_scale * log2(e)
    int out_f32;
    int chunk_e4m3;              // chunk K/V are E4M3 bytes (initial prefill on FP8 K/V)
    // fused NVFP4 append of the chunk (null pool: attention only)
    uint8_t *pool;               // page-head records [num_pages][hkv][record]
    const int32_t *slot_mapping; // [q rows]
    int num_pages;
    float gscale;                // tensor scale: blocks are taken of x / gscale
    HeadScales hs;
    uint32_t wait_limit;         // polls before a wait gives up (kWaitLimit by default)
    // E4M3 chunks: tensor maps of the four E4M3 row sets as [rows][hkv][128]
    // bytes, 64-row boxes of one kv head in the 128-byte swizzle, for the
    // kernel that reads every key tile by TMA (filled by the launcher)
    CUtensorMap tm_k_prefix;
    CUtensorMap tm_v_prefix;
    CUtensorMap tm_k_chunk;
    CUtensorMap tm_v_chunk;
};

// New rows into the block-scaled FP8 cache.
struct BlockAppendParams {
    const void *k_new;           // [num_tokens][hkv][128]
    const void *v_new;
    const int32_t *q_indptr;     // [batch + 1]: rows of each sequence
    const int32_t *block_table;  // [batch][max_pages]
    const int32_t *seq_lens;     // [batch], the new tokens included
    uint8_t *pool;               // page-head records [num_pages][hkv][kFp8BlockRecord]
    int32_t *dev_status;
    int num_tokens;
    int batch;
    int hkv;
    int max_pages;
    int num_pages;
    int in_bf16;
};

// Cached rows of the block-scaled FP8 cache, read back.
struct BlockReadParams {
    const uint8_t *pool;
    const int32_t *block_table;
    const int32_t *lens;         // [batch]
    const int32_t *kv_indptr;    // [batch] first output row of each sequence
    void *k_out;                 // [rows][hkv][128] of out_dtype
    void *v_out;
    int32_t *dev_status;
    int batch;
    int hkv;
    int max_pages;
    int num_pages;
    int out_dtype;               // nvfp4kv_dtype
};

// Bounds of the pages' keys.
struct BoundsParams {
    const uint8_t *pool;
    const int32_t *block_table;
    const int32_t *from_lens;    // [batch] or null: 0
    const int32_t *seq_lens;     // [batch]
    int8_t *bounds;              // [num_pages][hkv][2][128]: least, largest
    float *steps;                // [num_pages][hkv]
    int32_t *dev_status;
    int batch;
    int hkv;
    int max_pages;
    int num_pages;
};

// The pages that each query token looks at.
struct SelectParams {
    const int8_t *bounds;
    const float *steps;
    const uint16_t *q;           // bf16 [batch][q_len][hq][128]
    const int32_t *block_table;
    const int32_t *seq_lens;
    int32_t *pages;              // [batch][q_len][hkv][budget]
    int32_t *dev_status;
    int batch;
    int q_len;
    int hq;
    int hkv;
    int group;
    int max_pages;
    int num_pages;
    int budget;
    int first;                   // pages always taken, at the beginning
    int last;                    // ... and at the end
    int chunk_tiles;             // (set by the launcher) tiles of 16 pages a CTA has at most
    long long unit0;             // (set by the launcher) its first (query token, kv head)
};

// Chunk attention over the paged NVFP4 cache.
struct PagedExtendParams {
    const uint8_t *pool;         // page-head records
    const uint16_t *q;           // bf16 [q_rows][hq][128]
    const int32_t *q_indptr;     // [batch + 1]
    const int32_t *block_table;  // [batch][max_pages]
    const int32_t *seq_lens;     // [batch], the chunk's tokens included
    void *out;                   // [q_rows][hq][128], bf16 or fp32
    float *partials;             // workers > 1: two pieces and a note of each CTA (paged_extend.cu)
    int32_t *dev_status;
    int batch;
    int hq;
    int hkv;
    int group;
    int max_pages;
    int num_pages;
    int q_rows;
    int max_q_len;
    int window;                  // 0: none
    int workers;                 // CTAs (set by the launcher)
    int out_f32;
    float qscale;                // sm_scale * log2(e)
    float gscale;
    HeadScales hs;
    uint32_t wait_limit;
};

// How a paged extend call is cut: whether a CTA's two MMA blocks share their
// rows (and halve the keys), how many CTAs take part, and the bytes of
// workspace.
struct ExtendShape {
    bool key_split;
    int workers;
    size_t workspace;
};

// Head norm and rotation of new queries and keys; with a pool the keys and
// values go into the NVFP4 cache instead of k_out.
struct NormRopeParams {
    const void *q;               // rows [token][hq][128] at a token stride, in_dtype
    const void *k;
    const void *v;               // (append)
    int64_t q_stride;            // elements from one token to the next
    int64_t k_stride;
    int64_t v_stride;
    const int32_t *positions;    // [tokens], < 0: no such token
    const void *q_weight;        // [128] or null: no norm
    const void *k_weight;
    uint16_t *q_out;             // bf16 [tokens][hq][128]
    void *k_out;                 // [tokens][hkv][128], in_dtype
    uint8_t *pool;               // append: page-head records
    const int32_t *slot_mapping;
    int32_t *dev_status;
    int num_tokens;
    int hq;
    int hkv;
    int num_pages;
    int in_bf16;
    int weight_bf16;
    int rot;                     // rotated channels, a multiple of 32
    int interleaved;
    float eps;
    float rope_scale;            // multiplies cos and sin
    float gscale;
    int q_quads, quads;          // set by the launcher: fours of a token's query heads, and of all heads,
    long long v_jobs;            // and warps of V blocks
    HeadScales hs;
    uint64_t freq[kHeadDim / 2]; // turns a position, in units of 2^-64
    uint32_t wait_limit;
};

// A step's tables (plan: a = context lengths, b = new tokens) or the return of
// pages (release: a = old lengths, b = lengths kept).
struct StepTablesParams {
    const int32_t *lens_a;       // [batch]
    const int32_t *lens_b;       // [batch]
    int32_t *block_table;        // [batch][max_pages]
    const int32_t *free_pages;   // stack of free page ids, its top at num_free - 1 (plan)
    int32_t *free_pages_out;     // the same (release)
    const int32_t *num_free_in;
    int32_t *num_free_out;       // may be num_free_in
    int32_t *seq_lens;           // [batch]
    int32_t *q_indptr;           // [batch + 1]
    int32_t *kv_indptr;          // [batch], nullable
    int32_t *slot_mapping;       // [max_tokens]
    int32_t *positions;          // [max_tokens], nullable
    int32_t *dev_status;
    int batch;
    int max_pages;
    int num_pages;
    int free_capacity;
    int max_tokens;
    int count_here;              // the kernel itself writes num_free_out (set by the launcher)
};

// Launch with programmatic stream serialisation allowed, so the kernel's
// prologue may overlap the tail of the previous kernel in the stream; every
// kernel launched this way calls pdl_wait() before touching data that the
// previous kernel may still write or read.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}

// Allows a kernel the most dynamic shared memory that it can have beside
// kStatic bytes of its own, once a device: what is allowed is one for all threads, so a
// call's own need, set at each launch, might be taken back by another's before it starts
// (and the runtime call costs a launch a third of a microsecond).
template <auto kKernel, int kStatic = 0>
cudaError_t allow_shared()
{
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)))
        return e;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - kStatic);
    if (e == cudaSuccess && dev >= 0 && dev < 64)
        done[dev].store(true, std::memory_order_release);
    return e;
}

int sm_count();                  // current device, cached
int default_num_workers();       // sm_count * kDecodeCtasPerSm * kDecodeWarps
size_t decode_workspace_bytes(int num_workers);

cudaError_t launch_quantize_append_nvfp4(const QuantParams &p, cudaStream_t s);
cudaError_t launch_quantize_append_fp8(const QuantParams &p, cudaStream_t s);
cudaError_t launch_decode_nvfp4(const DecodeParams &p, cudaStream_t s);
cudaError_t launch_decode_nvfp4_multi(const DecodeParams &p, cudaStream_t s);
cudaError_t launch_decode_fp8(const DecodeParams &p, cudaStream_t s);
cudaError_t launch_decode_fp8_block(const DecodeParams &p, cudaStream_t s);         // (p.q_len > 1: several tokens)
cudaError_t launch_decode_selected_nvfp4(const DecodeParams &p, cudaStream_t s);
cudaError_t launch_decode_selected_fp8_block(const DecodeParams &p, cudaStream_t s);
// How clusters take a decode of so many (query token, kv head)s of at most so many pages.
struct ClusterPlan {
    int first = 0;               // (query token, kv head)s of the first launch; 0: the worker split
    int ranks = 1, rest_ranks = 1;
};
ClusterPlan plan_cluster_decode(int64_t segments, int64_t worker_segments, int64_t pages, bool eight_bits, bool listed,
                                int q_len);
cudaError_t launch_cluster_decode_nvfp4(const DecodeParams &p, const ClusterPlan &plan, cudaStream_t s);
cudaError_t launch_cluster_decode_fp8_block(const DecodeParams &p, const ClusterPlan &plan,
                                            cudaStream_t s);        // (listed or all pages)
cudaError_t launch_merge(const DecodeParams &p, cudaStream_t s);
cudaError_t launch_block_append(const BlockAppendParams &p, cudaStream_t s);
cudaError_t launch_block_read(const BlockReadParams &p, cudaStream_t s);
cudaError_t launch_page_bounds_nvfp4(const BoundsParams &p, cudaStream_t s);
cudaError_t launch_page_bounds_fp8_block(const BoundsParams &p, cudaStream_t s);
cudaError_t launch_select_pages(const SelectParams &p, cudaStream_t s);
cudaError_t launch_dequant_prefix_fp8(const PrefixParams &p, cudaStream_t s);
ExtendShape paged_extend_shape(int64_t q_rows, int64_t max_q_len, int64_t batch, int64_t hkv, int64_t group,
                               int64_t max_pages, int64_t window);
cudaError_t launch_paged_extend(const PagedExtendParams &p, const ExtendShape &shape, cudaStream_t s);
cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t s);    // appends when p.pool != null
cudaError_t launch_plan_step(const StepTablesParams &p, cudaStream_t s);
cudaError_t launch_release_pages(const StepTablesParams &p, cudaStream_t s);
cudaError_t launch_extend_attention(const ExtendParams &p, cudaStream_t s);   // appends when p.pool != null

} // namespace nvfp4kv
