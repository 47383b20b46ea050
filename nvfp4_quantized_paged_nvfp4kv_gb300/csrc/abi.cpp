// C ABI of the library: argument validation and launches.
// The contract of every entry point is documented in include/nvfp4kv.h.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "nvfp4kv.h"
#include "nvfp4kv_internal.h"

using namespace nvfp4kv;

namespace {

std::atomic<uint32_t> g_wait_limit{kWaitLimit};

uint32_t wait_limit()
{
    return g_wait_limit.load(std::memory_order_relaxed);
}

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

cudaStream_t to_cuda(nvfp4kv_stream_t s)
{
    return reinterpret_cast<cudaStream_t>(s);
}

nvfp4kv_status from_cuda(cudaError_t e)
{
    return e == cudaSuccess ? NVFP4KV_OK : NVFP4KV_ERR_CUDA;
}

bool normal_positive(float x)
{
    return x >= 1.17549435e-38f && x <= 3.40282347e+38f;
}

// Per-head tensor scales of a (checked) NVFP4 cache: fl32(G * factor) per kv
// head of K and V, or per_head = 0 without factors.
HeadScales head_scales_of(const nvfp4kv_cache *c)
{
    HeadScales hs{};
    if (c->head_scales == nullptr)
        return hs;
    hs.per_head = 1;
    for (int h = 0; h < c->num_kv_heads; ++h) {
        hs.k[h] = c->global_scale * c->head_scales[h];
        hs.v[h] = c->global_scale * c->head_scales[c->num_kv_heads + h];
    }
    return hs;
}

// Shared geometry checks for both cache kinds.
nvfp4kv_status check_geometry(int32_t num_pages, int32_t hkv, int32_t page_size, int32_t head_dim)
{
    if (num_pages <= 0 || hkv <= 0 || page_size <= 0 || head_dim <= 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (page_size != kPageSize || head_dim != kHeadDim)
        return NVFP4KV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(num_pages) * hkv > (int64_t{1} << 31) - 1)
        return NVFP4KV_ERR_UNSUPPORTED;
    return NVFP4KV_OK;
}

nvfp4kv_status check_nvfp4(const nvfp4kv_cache *c)
{
    if (c == nullptr)
        return NVFP4KV_ERR_INVALID_ARG;
    nvfp4kv_status st = check_geometry(c->num_pages, c->num_kv_heads, c->page_size, c->head_dim);
    if (st != NVFP4KV_OK)
        return st;
    // a positive, normal, finite tensor scale
    if (!normal_positive(c->global_scale))
        return NVFP4KV_ERR_UNSUPPORTED;
    // optional per-head factors: each, and its product with G, positive normal
    if (c->head_scales != nullptr) {
        if (c->num_kv_heads > kMaxScaledHeads)
            return NVFP4KV_ERR_UNSUPPORTED;
        for (int i = 0; i < 2 * c->num_kv_heads; ++i) {
            const float f = c->head_scales[i];
            if (!normal_positive(f) || !normal_positive(c->global_scale * f))
                return NVFP4KV_ERR_UNSUPPORTED;
        }
    }
    if (c->pool == nullptr || !aligned16(c->pool))
        return NVFP4KV_ERR_INVALID_ARG;
    return NVFP4KV_OK;
}

template <class Cache>                           // fp8kv_cache, fp8bkv_cache
nvfp4kv_status check_fp8(const Cache *c)
{
    if (c == nullptr)
        return NVFP4KV_ERR_INVALID_ARG;
    nvfp4kv_status st = check_geometry(c->num_pages, c->num_kv_heads, c->page_size, c->head_dim);
    if (st != NVFP4KV_OK)
        return st;
    if (c->pool == nullptr || !aligned16(c->pool))
        return NVFP4KV_ERR_INVALID_ARG;
    return NVFP4KV_OK;
}

nvfp4kv_status check_append(const void *k_new, const void *v_new, nvfp4kv_dtype in_dtype, int32_t num_tokens,
                            const int32_t *slot_mapping)
{
    if (num_tokens < 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (in_dtype != NVFP4KV_F32 && in_dtype != NVFP4KV_BF16)
        return NVFP4KV_ERR_INVALID_ARG;
    if (num_tokens == 0)
        return NVFP4KV_OK;
    if (k_new == nullptr || v_new == nullptr || slot_mapping == nullptr)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || (reinterpret_cast<uintptr_t>(slot_mapping) & 3u))
        return NVFP4KV_ERR_INVALID_ARG;
    return NVFP4KV_OK;
}

// Decode arguments common to both cache kinds.  Fills p (except the cache
// pointers) on success.
nvfp4kv_status check_decode(int32_t hkv, int32_t num_pages, const void *q, int32_t batch, int32_t num_q_heads,
                            const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
                            float sm_scale, void *out, nvfp4kv_dtype out_dtype, void *workspace,
                            size_t workspace_bytes, int32_t num_workers, int32_t *dev_status, DecodeParams &p)
{
    if (batch < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 || num_workers < 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (out_dtype != NVFP4KV_F32 && out_dtype != NVFP4KV_BF16)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!std::isfinite(sm_scale))
        return NVFP4KV_ERR_INVALID_ARG;
    if (num_q_heads % hkv != 0)
        return NVFP4KV_ERR_INVALID_ARG;
    const int group = num_q_heads / hkv;
    if (group > kMaxGroup)
        return NVFP4KV_ERR_UNSUPPORTED;
    if (batch > kMaxBatch)
        return NVFP4KV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(batch) * hkv * max_pages_per_seq > (int64_t{1} << 31) - 1)
        return NVFP4KV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_pages_per_seq) * kPageSize > (int64_t{1} << 30))
        return NVFP4KV_ERR_UNSUPPORTED;
    if (batch > 0) {
        if (q == nullptr || out == nullptr || block_table == nullptr || seq_lens == nullptr)
            return NVFP4KV_ERR_INVALID_ARG;
        if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
            (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
            return NVFP4KV_ERR_INVALID_ARG;
    }
    int nw = num_workers;
    if (nw == 0) {
        // automatic: the device default, but no more than one worker per four
        // page-heads of the largest possible batch
        const int64_t upper = static_cast<int64_t>(batch) * hkv * max_pages_per_seq;
        int64_t cap = upper / 4;
        if (cap < 1)
            cap = 1;
        nw = default_num_workers();
        if (nw > cap)
            nw = static_cast<int>(cap);
    }
    if (batch > 0) {
        if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u))
            return NVFP4KV_ERR_WORKSPACE;
        if (workspace_bytes < decode_workspace_bytes(nw))
            return NVFP4KV_ERR_WORKSPACE;
    }
    p = DecodeParams{};
    p.q = static_cast<const uint16_t *>(q);
    p.out = out;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.dev_status = dev_status;
    p.partials = static_cast<float *>(workspace);
    p.batch = batch;
    p.hq = num_q_heads;
    p.hkv = hkv;
    p.group = group;
    p.max_pages = max_pages_per_seq;
    p.num_pages = num_pages;
    p.out_bf16 = out_dtype == NVFP4KV_BF16;
    p.num_workers = nw;
    p.qscale = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
    p.out_scale = 1.f;
    p.gscale = 1.f;
    p.q_len = 1;
    p.rows = group;
    p.row_groups = 1;
    p.lanes = 1;
    p.wait_limit = wait_limit();
    return NVFP4KV_OK;
}

// The NVFP4 tensor scale G: scores see G * k, so G joins the query scale;
// outputs see G * v, so the normaliser carries it.  With per-head factors each
// kv head has its own query scale, append divisors and output scale.
void apply_tensor_scale(DecodeParams &p, float sm_scale, const nvfp4kv_cache *c)
{
    const float G = c->global_scale;
    p.qscale = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634 * static_cast<double>(G));
    p.out_scale = G;
    p.gscale = G;
    p.hs = head_scales_of(c);
    if (p.hs.per_head)
        for (int h = 0; h < c->num_kv_heads; ++h)
            p.qs[h] = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634 *
                                         static_cast<double>(p.hs.k[h]));
}

// Extend arguments common to both entry points.  Fills p (attention part)
// on success; batch == 0 or max_q_len == 0 is valid and launches nothing.
nvfp4kv_status check_extend(const void *q, const int32_t *q_indptr, int32_t q_rows, int32_t max_q_len,
                            const void *k_prefix, const void *v_prefix, const int32_t *kv_indptr,
                            const int32_t *prefix_lens, int64_t prefix_rows, const void *k_chunk,
                            const void *v_chunk, nvfp4kv_dtype chunk_dtype, int32_t batch, int32_t num_q_heads,
                            int32_t num_kv_heads, float sm_scale, void *out, nvfp4kv_dtype out_dtype,
                            int32_t *dev_status, ExtendParams &p)
{
    if (batch < 0 || q_rows < 0 || max_q_len < 0 || prefix_rows < 0 || num_q_heads <= 0 || num_kv_heads <= 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (out_dtype != NVFP4KV_F32 && out_dtype != NVFP4KV_BF16)
        return NVFP4KV_ERR_INVALID_ARG;
    if (chunk_dtype != NVFP4KV_BF16 && chunk_dtype != NVFP4KV_E4M3)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!std::isfinite(sm_scale))
        return NVFP4KV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0)
        return NVFP4KV_ERR_INVALID_ARG;
    const int group = num_q_heads / num_kv_heads;
    if (group > kMaxGroup || num_kv_heads > 65535 || batch > 65535)
        return NVFP4KV_ERR_UNSUPPORTED;
    // rows of one sequence and kv head (chunk length x group) stay within
    // int32; workspace element offsets within int64
    if (static_cast<int64_t>(max_q_len) * group > (int64_t{1} << 31) - kMaxGroup * 128)
        return NVFP4KV_ERR_UNSUPPORTED;
    if (prefix_rows > (int64_t{1} << 40) / (static_cast<int64_t>(num_kv_heads) * kHeadDim))
        return NVFP4KV_ERR_UNSUPPORTED;
    if (batch == 0 || max_q_len == 0)
        return NVFP4KV_OK;
    if (q == nullptr || q_indptr == nullptr || kv_indptr == nullptr || prefix_lens == nullptr || k_chunk == nullptr ||
        v_chunk == nullptr || out == nullptr)
        return NVFP4KV_ERR_INVALID_ARG;
    if (prefix_rows > 0 && (k_prefix == nullptr || v_prefix == nullptr))
        return NVFP4KV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_chunk) || !aligned16(v_chunk) || !aligned16(out) || !aligned16(k_prefix) ||
        !aligned16(v_prefix) || (reinterpret_cast<uintptr_t>(q_indptr) & 3u) ||
        (reinterpret_cast<uintptr_t>(kv_indptr) & 3u) || (reinterpret_cast<uintptr_t>(prefix_lens) & 3u))
        return NVFP4KV_ERR_INVALID_ARG;
    p = ExtendParams{};
    p.q = static_cast<const uint16_t *>(q);
    p.q_indptr = q_indptr;
    p.k_prefix = static_cast<const uint8_t *>(k_prefix);
    p.v_prefix = static_cast<const uint8_t *>(v_prefix);
    p.kv_indptr = kv_indptr;
    p.prefix_lens = prefix_lens;
    p.k_chunk = k_chunk;
    p.v_chunk = v_chunk;
    p.chunk_e4m3 = chunk_dtype == NVFP4KV_E4M3;
    p.out = out;
    p.dev_status = dev_status;
    p.batch = batch;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.group = group;
    p.q_rows = q_rows;
    p.max_q_len = max_q_len;
    p.prefix_rows = prefix_rows;
    p.qscale = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
    p.out_f32 = out_dtype == NVFP4KV_F32;
    p.gscale = 1.f;
    p.wait_limit = wait_limit();
    return NVFP4KV_OK;
}

// A caller's array, as the overlap checks see it.
struct Span {
    const void *p;
    size_t bytes;
    bool written;
};

// Whether an array that the call writes shares memory with another one.
template <size_t N>
bool written_overlap(const Span (&a)[N])
{
    for (size_t i = 0; i < N; ++i)
        for (size_t j = i + 1; j < N; ++j) {
            if (!(a[i].written || a[j].written) || a[i].p == nullptr || a[j].p == nullptr || a[i].bytes == 0 ||
                a[j].bytes == 0)
                continue;
            const uintptr_t x = reinterpret_cast<uintptr_t>(a[i].p), y = reinterpret_cast<uintptr_t>(a[j].p);
            if (x < y ? y - x < a[i].bytes : x - y < a[j].bytes)
                return true;
        }
    return false;
}

bool aligned4(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

// Checks that plan_step and release_pages share.
nvfp4kv_status check_tables(const int32_t *a, const int32_t *b, int32_t batch, const int32_t *block_table,
                            int32_t max_pages_per_seq, int32_t num_pages, const int32_t *free_pages,
                            int32_t free_capacity, const int32_t *num_free_in, const int32_t *num_free_out)
{
    if (batch < 0 || max_pages_per_seq <= 0 || num_pages <= 0 || free_capacity < 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (batch > kMaxBatch || static_cast<int64_t>(batch) * max_pages_per_seq > (int64_t{1} << 31) - 1 ||
        static_cast<int64_t>(max_pages_per_seq) * kPageSize > (int64_t{1} << 30) ||
        static_cast<int64_t>(num_pages) * kPageSize > (int64_t{1} << 31) - 1)
        return NVFP4KV_ERR_UNSUPPORTED;
    if (batch > 0 && (a == nullptr || b == nullptr || block_table == nullptr))
        return NVFP4KV_ERR_INVALID_ARG;
    if (num_free_in == nullptr || num_free_out == nullptr || (free_capacity > 0 && free_pages == nullptr))
        return NVFP4KV_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(a), static_cast<const void *>(b),
                          static_cast<const void *>(block_table), static_cast<const void *>(free_pages),
                          static_cast<const void *>(num_free_in), static_cast<const void *>(num_free_out)})
        if (!aligned4(p))
            return NVFP4KV_ERR_INVALID_ARG;
    return NVFP4KV_OK;
}

// Sizes of a paged extend call.
nvfp4kv_status check_paged_extend_sizes(int32_t q_rows, int32_t max_q_len, int32_t batch, int32_t hq, int32_t hkv,
                                        int32_t max_pages, int32_t window)
{
    if (q_rows < 0 || max_q_len < 0 || batch < 0 || hq <= 0 || hkv <= 0 || max_pages <= 0 || window < 0 || hq % hkv != 0)
        return NVFP4KV_ERR_INVALID_ARG;
    const int64_t group = hq / hkv;
    if (group > kMaxGroup || hkv > 65535 || batch > kMaxBatch || max_q_len * group >= (int64_t{1} << 30) ||
        static_cast<int64_t>(max_pages) * kPageSize > (int64_t{1} << 30))
        return NVFP4KV_ERR_UNSUPPORTED;
    return NVFP4KV_OK;
}

// A block table, the lengths of its rows, and an optional array as long.
nvfp4kv_status check_rows(int32_t batch, const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *lens,
                          const int32_t *more)
{
    if (batch < 0 || max_pages_per_seq <= 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (batch > kMaxBatch || static_cast<int64_t>(batch) * max_pages_per_seq > (int64_t{1} << 31) - 1 ||
        static_cast<int64_t>(max_pages_per_seq) * kPageSize > (int64_t{1} << 30))
        return NVFP4KV_ERR_UNSUPPORTED;
    if (batch > 0 && (block_table == nullptr || lens == nullptr || !aligned4(block_table) || !aligned4(lens) ||
                      !aligned4(more)))
        return NVFP4KV_ERR_INVALID_ARG;
    return NVFP4KV_OK;
}

nvfp4kv_status check_bounds(const nvfp4kv_bounds *b)
{
    if (b == nullptr || b->num_pages <= 0 || b->num_kv_heads <= 0 || b->bounds == nullptr || !aligned16(b->bounds) ||
        b->steps == nullptr || !aligned4(b->steps))
        return NVFP4KV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(b->num_pages) * b->num_kv_heads > (int64_t{1} << 31) - 1)
        return NVFP4KV_ERR_UNSUPPORTED;
    return NVFP4KV_OK;
}

size_t heads_of(const nvfp4kv_bounds *b)
{
    return static_cast<size_t>(b->num_pages) * b->num_kv_heads;
}

// Bounds of either cache's pages; the cache is checked.
template <class Cache, class Launch>
nvfp4kv_status page_bounds(const Cache *cache, size_t record, const nvfp4kv_bounds *bounds, const int32_t *block_table,
                           int32_t max_pages_per_seq, const int32_t *from_lens, const int32_t *seq_lens, int32_t batch,
                           int32_t *dev_status, nvfp4kv_stream_t stream, Launch launch)
{
    nvfp4kv_status st = check_bounds(bounds);
    if (st != NVFP4KV_OK)
        return st;
    if (bounds->num_pages != cache->num_pages || bounds->num_kv_heads != cache->num_kv_heads)
        return NVFP4KV_ERR_INVALID_ARG;
    st = check_rows(batch, block_table, max_pages_per_seq, seq_lens, from_lens);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    const size_t n = 4 * static_cast<size_t>(batch), heads = heads_of(bounds);
    const Span spans[] = {{cache->pool, heads * record, false},
                          {block_table, n * static_cast<size_t>(max_pages_per_seq), false},
                          {from_lens, n, false},
                          {seq_lens, n, false},
                          {bounds->bounds, heads * 2 * kHeadDim, true},
                          {bounds->steps, 4 * heads, true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    BoundsParams p{};
    p.pool = static_cast<const uint8_t *>(cache->pool);
    p.block_table = block_table;
    p.from_lens = from_lens;
    p.seq_lens = seq_lens;
    p.bounds = bounds->bounds;
    p.steps = bounds->steps;
    p.dev_status = dev_status;
    p.batch = batch;
    p.hkv = cache->num_kv_heads;
    p.max_pages = max_pages_per_seq;
    p.num_pages = cache->num_pages;
    return from_cuda(launch(p, to_cuda(stream)));
}

constexpr int32_t kMaxSelectPages = NVFP4KV_MAX_SELECT_PAGES;

nvfp4kv_status check_query_tokens(int32_t batch, int32_t q_len)
{
    if (batch < 0 || q_len < 1)
        return NVFP4KV_ERR_INVALID_ARG;
    if (q_len > NVFP4KV_MAX_QUERY_TOKENS || static_cast<int64_t>(batch) * q_len > kMaxBatch)
        return NVFP4KV_ERR_UNSUPPORTED;
    return NVFP4KV_OK;
}

nvfp4kv_status check_select_sizes(int32_t batch, int32_t q_len, int32_t hkv, int32_t max_pages)
{
    const nvfp4kv_status st = check_query_tokens(batch, q_len);
    if (st != NVFP4KV_OK)
        return st;
    if (hkv <= 0 || max_pages <= 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (max_pages > kMaxSelectPages || static_cast<int64_t>(batch) * q_len * hkv > (int64_t{1} << 27))
        return NVFP4KV_ERR_UNSUPPORTED;
    return NVFP4KV_OK;
}

// How clusters take a decode over listed pages (none of it: the worker split).
ClusterPlan cluster_plan(const DecodeParams &p, bool eight_bits)
{
    const int64_t segments = static_cast<int64_t>(p.batch) * p.hkv;
    return plan_cluster_decode(segments, segments, p.budget < p.max_pages ? p.budget : p.max_pages, eight_bits, true,
                               p.sel_q_len);
}

// Decode over listed pages: fills p (except the cache's pool and scales).
nvfp4kv_status check_selected(int32_t hkv, int32_t num_pages, size_t pool_bytes, const void *pool, const void *q,
                              int32_t batch, int32_t q_len, int32_t num_q_heads, const int32_t *block_table,
                              int32_t max_pages_per_seq, const int32_t *seq_lens, const int32_t *pages, int32_t budget,
                              float sm_scale, void *out, nvfp4kv_dtype out_dtype, void *workspace,
                              size_t workspace_bytes, int32_t num_workers, int32_t *dev_status, DecodeParams &p)
{
    nvfp4kv_status st = check_query_tokens(batch, q_len);
    if (st != NVFP4KV_OK)
        return st;
    st = check_rows(batch, block_table, max_pages_per_seq, seq_lens, pages);
    if (st != NVFP4KV_OK)
        return st;
    if (budget <= 0)
        return NVFP4KV_ERR_INVALID_ARG;
    // (a row's pages are at most the budget: what the work split is made for)
    const int32_t most = budget < max_pages_per_seq ? budget : max_pages_per_seq;
    st = check_decode(hkv, num_pages, q, batch * q_len, num_q_heads, block_table, most, seq_lens, sm_scale, out,
                      out_dtype, workspace, workspace_bytes, num_workers, dev_status, p);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    if (pages == nullptr)
        return NVFP4KV_ERR_INVALID_ARG;
    const size_t rows = static_cast<size_t>(batch) * q_len, elems = rows * num_q_heads * kHeadDim;
    const Span spans[] = {{q, 2 * elems, false},
                          {block_table, 4 * static_cast<size_t>(batch) * max_pages_per_seq, false},
                          {seq_lens, 4 * static_cast<size_t>(batch), false},
                          {pages, 4 * rows * hkv * static_cast<size_t>(budget), false},
                          {pool, pool_bytes, false},
                          {out, elems * (out_dtype == NVFP4KV_F32 ? 4 : 2), true},
                          {workspace, decode_workspace_bytes(p.num_workers), true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    p.max_pages = max_pages_per_seq;
    p.sel_pages = pages;
    p.budget = budget;
    p.sel_q_len = q_len;
    return NVFP4KV_OK;
}

// Rows of `heads` x 128 channels at a token stride: base and stride keep every
// row on 16 bytes, and rows do not overlap.
bool good_rows(const void *base, int64_t stride, int32_t heads, int elem_bytes)
{
    return base != nullptr && aligned16(base) && stride >= static_cast<int64_t>(heads) * kHeadDim &&
           stride <= (int64_t{1} << 28) && (stride * elem_bytes) % 16 == 0;
}

size_t rows_bytes(int64_t stride, int32_t tokens, int32_t heads, int elem_bytes)
{
    return (static_cast<size_t>(stride) * (tokens - 1) + static_cast<size_t>(heads) * kHeadDim) * elem_bytes;
}

// f / 2 pi modulo 1 in units of 2^-64: |f| times 1 / 2 pi held as the sum of
// two doubles (the product is good to about 2^-105 of itself before the whole
// turns go), negated modulo 2^64 for a negative f.
uint64_t turn_fraction(double f)
{
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double a = std::fabs(f);
    const double hi = a * kHi, lo = std::fma(a, kHi, -hi) + a * kLo;
    const double rest = std::ldexp(lo, 64);           // below 2^62 while a is below 2^49; past that no fraction is left
    uint64_t turn = static_cast<uint64_t>(std::ldexp(hi - std::floor(hi), 64));
    if (std::fabs(rest) < 0x1p62)
        turn += static_cast<uint64_t>(static_cast<int64_t>(rest));
    return f < 0.0 ? uint64_t{0} - turn : turn;
}

// Arguments that the two norm-and-rotation calls share.  Fills p on success;
// num_tokens == 0 is valid and launches nothing.
nvfp4kv_status check_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                               nvfp4kv_dtype in_dtype, int32_t num_tokens, int32_t num_q_heads,
                               int32_t num_kv_heads, const int32_t *positions, const nvfp4kv_rope *rope,
                               const nvfp4kv_head_norm *norm, void *q_out, NormRopeParams &p)
{
    if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (in_dtype != NVFP4KV_F32 && in_dtype != NVFP4KV_BF16)
        return NVFP4KV_ERR_INVALID_ARG;
    if (num_q_heads > 65535 || num_kv_heads > 65535)
        return NVFP4KV_ERR_UNSUPPORTED;
    p = NormRopeParams{};
    p.rope_scale = 1.f;
    if (rope != nullptr) {
        if (rope->rotary_dim < 0 || rope->rotary_dim > kHeadDim || rope->rotary_dim % 32 != 0 ||
            (rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite(rope->scale))
            return NVFP4KV_ERR_UNSUPPORTED;
        if (rope->rotary_dim > 0 && rope->inv_freq == nullptr)
            return NVFP4KV_ERR_INVALID_ARG;
        for (int i = 0; i < rope->rotary_dim / 2; ++i) {
            if (!std::isfinite(rope->inv_freq[i]))
                return NVFP4KV_ERR_UNSUPPORTED;
            p.freq[i] = turn_fraction(rope->inv_freq[i]);
        }
        p.rot = rope->rotary_dim;
        p.interleaved = rope->interleaved;
        p.rope_scale = rope->scale;
    }
    if (norm != nullptr) {
        if (norm->weight_dtype != NVFP4KV_F32 && norm->weight_dtype != NVFP4KV_BF16)
            return NVFP4KV_ERR_INVALID_ARG;
        if (!std::isfinite(norm->eps) || norm->eps < 0.f)
            return NVFP4KV_ERR_UNSUPPORTED;
        const uintptr_t mask = norm->weight_dtype == NVFP4KV_F32 ? 3u : 1u;
        if ((reinterpret_cast<uintptr_t>(norm->q_weight) & mask) || (reinterpret_cast<uintptr_t>(norm->k_weight) & mask))
            return NVFP4KV_ERR_INVALID_ARG;
        p.q_weight = norm->q_weight;
        p.k_weight = norm->k_weight;
        p.weight_bf16 = norm->weight_dtype == NVFP4KV_BF16;
        p.eps = norm->eps;
    }
    if (num_tokens == 0)
        return NVFP4KV_OK;
    const int size = in_dtype == NVFP4KV_BF16 ? 2 : 4;
    if (!good_rows(q, q_stride, num_q_heads, size) || !good_rows(k, k_stride, num_kv_heads, size) ||
        q_out == nullptr || !aligned16(q_out) || positions == nullptr || !aligned4(positions))
        return NVFP4KV_ERR_INVALID_ARG;
    p.q = q;
    p.k = k;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.positions = positions;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.num_tokens = num_tokens;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.in_bf16 = in_dtype == NVFP4KV_BF16;
    p.wait_limit = wait_limit();
    return NVFP4KV_OK;
}

} // namespace

extern "C" {

nvfp4kv_status nvfp4kv_quantize_append(const nvfp4kv_cache *cache, const void *k_new, const void *v_new,
                                       nvfp4kv_dtype in_dtype, int32_t num_tokens, const int32_t *slot_mapping,
                                       int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_nvfp4(cache);
    if (st != NVFP4KV_OK)
        return st;
    st = check_append(k_new, v_new, in_dtype, num_tokens, slot_mapping);
    if (st != NVFP4KV_OK || num_tokens == 0)
        return st;
    QuantParams p{};
    p.k_new = k_new;
    p.v_new = v_new;
    p.slot_mapping = slot_mapping;
    p.pool = static_cast<uint8_t *>(cache->pool);
    p.dev_status = dev_status;
    p.num_tokens = num_tokens;
    p.hkv = cache->num_kv_heads;
    p.num_pages = cache->num_pages;
    p.in_bf16 = in_dtype == NVFP4KV_BF16;
    p.gscale = cache->global_scale;
    p.hs = head_scales_of(cache);
    return from_cuda(launch_quantize_append_nvfp4(p, to_cuda(stream)));
}

size_t nvfp4kv_decode_workspace_size(int32_t num_workers)
{
    return decode_workspace_bytes(num_workers < 0 ? 0 : num_workers);
}

nvfp4kv_status nvfp4kv_paged_decode(const nvfp4kv_cache *cache, const void *q, int32_t batch,
                                    int32_t num_q_heads, const int32_t *block_table, int32_t max_pages_per_seq,
                                    const int32_t *seq_lens, float sm_scale, void *out, nvfp4kv_dtype out_dtype,
                                    void *workspace, size_t workspace_bytes, int32_t num_workers,
                                    int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_nvfp4(cache);
    if (st != NVFP4KV_OK)
        return st;
    DecodeParams p;
    st = check_decode(cache->num_kv_heads, cache->num_pages, q, batch, num_q_heads, block_table,
                      max_pages_per_seq, seq_lens, sm_scale, out, out_dtype, workspace, workspace_bytes,
                      num_workers, dev_status, p);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    p.pool = static_cast<const uint8_t *>(cache->pool);
    apply_tensor_scale(p, sm_scale, cache);
    cudaError_t e = launch_decode_nvfp4(p, to_cuda(stream));
    if (e == cudaSuccess)
        e = launch_merge(p, to_cuda(stream));
    return from_cuda(e);
}

nvfp4kv_status nvfp4kv_paged_decode_multi(const nvfp4kv_cache *cache, const void *q, int32_t batch, int32_t q_len,
                                          int32_t num_q_heads, const int32_t *block_table,
                                          int32_t max_pages_per_seq, const int32_t *seq_lens, float sm_scale,
                                          void *out, nvfp4kv_dtype out_dtype, void *workspace,
                                          size_t workspace_bytes, int32_t num_workers, int32_t *dev_status,
                                          nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_nvfp4(cache);
    if (st != NVFP4KV_OK)
        return st;
    if (q_len < 1 || q_len > NVFP4KV_MAX_QUERY_TOKENS)
        return q_len < 1 ? NVFP4KV_ERR_INVALID_ARG : NVFP4KV_ERR_UNSUPPORTED;
    DecodeParams p;
    st = check_decode(cache->num_kv_heads, cache->num_pages, q, batch, num_q_heads, block_table,
                      max_pages_per_seq, seq_lens, sm_scale, out, out_dtype, workspace, workspace_bytes,
                      num_workers, dev_status, p);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    p.q_len = q_len;
    p.rows = p.group * q_len;
    p.row_groups = (p.rows + kMaxGroup - 1) / kMaxGroup;
    if (static_cast<int64_t>(batch) * cache->num_kv_heads * p.row_groups * max_pages_per_seq >
        (int64_t{1} << 31) - 1)
        return NVFP4KV_ERR_UNSUPPORTED;
    p.pool = static_cast<const uint8_t *>(cache->pool);
    apply_tensor_scale(p, sm_scale, cache);
    cudaError_t e = launch_decode_nvfp4_multi(p, to_cuda(stream));
    if (e == cudaSuccess)
        e = launch_merge(p, to_cuda(stream));
    return from_cuda(e);
}

nvfp4kv_status nvfp4kv_dequant_prefix_fp8(const nvfp4kv_cache *cache, const int32_t *block_table,
                                          int32_t max_pages_per_seq, const int32_t *prefix_lens,
                                          const int32_t *kv_indptr, int32_t batch, void *k_fp8_out,
                                          void *v_fp8_out, int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_nvfp4(cache);
    if (st != NVFP4KV_OK)
        return st;
    if (batch < 0 || max_pages_per_seq <= 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_pages_per_seq) * kPageSize > (int64_t{1} << 30))
        return NVFP4KV_ERR_UNSUPPORTED;
    if (batch == 0)
        return NVFP4KV_OK;
    if (block_table == nullptr || prefix_lens == nullptr || kv_indptr == nullptr || k_fp8_out == nullptr ||
        v_fp8_out == nullptr)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!aligned16(k_fp8_out) || !aligned16(v_fp8_out) || (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
        (reinterpret_cast<uintptr_t>(prefix_lens) & 3u) || (reinterpret_cast<uintptr_t>(kv_indptr) & 3u))
        return NVFP4KV_ERR_INVALID_ARG;
    PrefixParams p{};
    p.pool = static_cast<const uint8_t *>(cache->pool);
    p.block_table = block_table;
    p.prefix_lens = prefix_lens;
    p.kv_indptr = kv_indptr;
    p.k_out = static_cast<uint8_t *>(k_fp8_out);
    p.v_out = static_cast<uint8_t *>(v_fp8_out);
    p.dev_status = dev_status;
    p.batch = batch;
    p.hkv = cache->num_kv_heads;
    p.max_pages = max_pages_per_seq;
    p.num_pages = cache->num_pages;
    p.gscale = cache->global_scale;
    p.hs = head_scales_of(cache);
    p.wait_limit = wait_limit();
    return from_cuda(launch_dequant_prefix_fp8(p, to_cuda(stream)));
}

nvfp4kv_status nvfp4kv_extend_attention_fp8(const void *q, const int32_t *q_indptr, int32_t q_rows,
                                            int32_t max_q_len, const void *k_prefix, const void *v_prefix,
                                            const int32_t *kv_indptr, const int32_t *prefix_lens,
                                            int64_t prefix_rows, const void *k_chunk, const void *v_chunk,
                                            nvfp4kv_dtype chunk_dtype, int32_t batch, int32_t num_q_heads,
                                            int32_t num_kv_heads, float sm_scale, void *out,
                                            nvfp4kv_dtype out_dtype, int32_t *dev_status, nvfp4kv_stream_t stream)
{
    ExtendParams p{};
    const nvfp4kv_status st =
        check_extend(q, q_indptr, q_rows, max_q_len, k_prefix, v_prefix, kv_indptr, prefix_lens, prefix_rows,
                     k_chunk, v_chunk, chunk_dtype, batch, num_q_heads, num_kv_heads, sm_scale, out, out_dtype,
                     dev_status, p);
    if (st != NVFP4KV_OK || batch == 0 || max_q_len == 0)
        return st;
    return from_cuda(launch_extend_attention(p, to_cuda(stream)));
}

nvfp4kv_status nvfp4kv_extend_attention_fp8_append(const nvfp4kv_cache *cache, const int32_t *slot_mapping,
                                                   const void *q, const int32_t *q_indptr, int32_t q_rows,
                                                   int32_t max_q_len, const void *k_prefix, const void *v_prefix,
                                                   const int32_t *kv_indptr, const int32_t *prefix_lens,
                                                   int64_t prefix_rows, const void *k_chunk, const void *v_chunk,
                                                   nvfp4kv_dtype chunk_dtype, int32_t batch, int32_t num_q_heads,
                                                   float sm_scale, void *out, nvfp4kv_dtype out_dtype,
                                                   int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_nvfp4(cache);
    if (st != NVFP4KV_OK)
        return st;
    ExtendParams p{};
    st = check_extend(q, q_indptr, q_rows, max_q_len, k_prefix, v_prefix, kv_indptr, prefix_lens, prefix_rows,
                      k_chunk, v_chunk, chunk_dtype, batch, num_q_heads, cache->num_kv_heads, sm_scale, out,
                      out_dtype, dev_status, p);
    if (st != NVFP4KV_OK || batch == 0 || max_q_len == 0)
        return st;
    if (slot_mapping == nullptr || (reinterpret_cast<uintptr_t>(slot_mapping) & 3u))
        return NVFP4KV_ERR_INVALID_ARG;
    p.pool = static_cast<uint8_t *>(cache->pool);
    p.slot_mapping = slot_mapping;
    p.num_pages = cache->num_pages;
    p.gscale = cache->global_scale;
    p.hs = head_scales_of(cache);
    return from_cuda(launch_extend_attention(p, to_cuda(stream)));
}

size_t nvfp4kv_paged_extend_workspace_size(int32_t q_rows, int32_t max_q_len, int32_t batch, int32_t num_q_heads,
                                           int32_t num_kv_heads, int32_t max_pages_per_seq, int32_t window)
{
    if (check_paged_extend_sizes(q_rows, max_q_len, batch, num_q_heads, num_kv_heads, max_pages_per_seq, window) !=
        NVFP4KV_OK)
        return 0;
    return paged_extend_shape(q_rows, max_q_len, batch, num_kv_heads, num_q_heads / num_kv_heads, max_pages_per_seq,
                              window >= max_pages_per_seq * kPageSize ? 0 : window)
        .workspace;
}

nvfp4kv_status nvfp4kv_paged_extend(const nvfp4kv_cache *cache, const void *q, const int32_t *q_indptr,
                                    int32_t q_rows, int32_t max_q_len, int32_t batch, int32_t num_q_heads,
                                    const int32_t *block_table, int32_t max_pages_per_seq,
                                    const int32_t *seq_lens, int32_t window, float sm_scale, void *out,
                                    nvfp4kv_dtype out_dtype, void *workspace, size_t workspace_bytes,
                                    int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_nvfp4(cache);
    if (st != NVFP4KV_OK)
        return st;
    st = check_paged_extend_sizes(q_rows, max_q_len, batch, num_q_heads, cache->num_kv_heads, max_pages_per_seq, window);
    if (st != NVFP4KV_OK)
        return st;
    if ((out_dtype != NVFP4KV_F32 && out_dtype != NVFP4KV_BF16) || !std::isfinite(sm_scale))
        return NVFP4KV_ERR_INVALID_ARG;
    if (batch == 0 || max_q_len == 0 || q_rows == 0)
        return NVFP4KV_OK;
    if (window >= max_pages_per_seq * kPageSize)
        window = 0;                              // no sequence is longer
    if (q == nullptr || out == nullptr || q_indptr == nullptr || block_table == nullptr || seq_lens == nullptr ||
        !aligned16(q) || !aligned16(out) || !aligned4(q_indptr) || !aligned4(block_table) || !aligned4(seq_lens))
        return NVFP4KV_ERR_INVALID_ARG;
    const int32_t group = num_q_heads / cache->num_kv_heads;
    const ExtendShape shape = paged_extend_shape(q_rows, max_q_len, batch, cache->num_kv_heads, group, max_pages_per_seq,
                                                 window);
    if (shape.workspace > 0 && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
                                workspace_bytes < shape.workspace))
        return NVFP4KV_ERR_WORKSPACE;
    const size_t elems = static_cast<size_t>(q_rows) * num_q_heads * kHeadDim;
    const Span spans[] = {{q, 2 * elems, false},
                          {q_indptr, 4 * (static_cast<size_t>(batch) + 1), false},
                          {block_table, 4 * static_cast<size_t>(batch) * max_pages_per_seq, false},
                          {seq_lens, 4 * static_cast<size_t>(batch), false},
                          {cache->pool, static_cast<size_t>(cache->num_pages) * cache->num_kv_heads * kNvfp4Record, false},
                          {out, elems * (out_dtype == NVFP4KV_F32 ? 4 : 2), true},
                          {workspace, shape.workspace, true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    PagedExtendParams p{};
    p.pool = static_cast<const uint8_t *>(cache->pool);
    p.q = static_cast<const uint16_t *>(q);
    p.q_indptr = q_indptr;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.out = out;
    p.partials = static_cast<float *>(workspace);
    p.dev_status = dev_status;
    p.batch = batch;
    p.hq = num_q_heads;
    p.hkv = cache->num_kv_heads;
    p.group = group;
    p.max_pages = max_pages_per_seq;
    p.num_pages = cache->num_pages;
    p.q_rows = q_rows;
    p.max_q_len = max_q_len;
    p.window = window;
    p.out_f32 = out_dtype == NVFP4KV_F32;
    p.qscale = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
    p.gscale = cache->global_scale;
    p.hs = head_scales_of(cache);
    p.wait_limit = wait_limit();
    return from_cuda(launch_paged_extend(p, shape, to_cuda(stream)));
}

nvfp4kv_status nvfp4kv_plan_step(const int32_t *context_lens, const int32_t *new_lens, int32_t batch,
                                 int32_t *block_table, int32_t max_pages_per_seq, int32_t num_pages,
                                 const int32_t *free_pages, int32_t free_capacity, const int32_t *num_free_in,
                                 int32_t *num_free_out, int32_t *seq_lens, int32_t *q_indptr, int32_t *kv_indptr,
                                 int32_t *slot_mapping, int32_t *positions, int32_t max_tokens,
                                 int32_t *dev_status, nvfp4kv_stream_t stream)
{
    const nvfp4kv_status st = check_tables(context_lens, new_lens, batch, block_table, max_pages_per_seq, num_pages,
                                           free_pages, free_capacity, num_free_in, num_free_out);
    if (st != NVFP4KV_OK)
        return st;
    if (max_tokens < 0 || q_indptr == nullptr || (batch > 0 && seq_lens == nullptr) ||
        (max_tokens > 0 && slot_mapping == nullptr))
        return NVFP4KV_ERR_INVALID_ARG;
    if (!aligned4(seq_lens) || !aligned4(q_indptr) || !aligned4(kv_indptr) || !aligned4(slot_mapping) ||
        !aligned4(positions))
        return NVFP4KV_ERR_INVALID_ARG;
    const size_t n = 4 * static_cast<size_t>(batch), t = 4 * static_cast<size_t>(max_tokens);
    const Span spans[] = {{context_lens, n, false},
                          {new_lens, n, false},
                          {free_pages, 4 * static_cast<size_t>(free_capacity), false},
                          {num_free_in, 4, false},
                          {num_free_out == num_free_in ? nullptr : num_free_out, 4, true},
                          {block_table, n * static_cast<size_t>(max_pages_per_seq), true},
                          {seq_lens, n, true},
                          {q_indptr, n + 4, true},
                          {kv_indptr, n, true},
                          {slot_mapping, t, true},
                          {positions, t, true},
                          {dev_status, 4, true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    StepTablesParams p{};
    p.lens_a = context_lens;
    p.lens_b = new_lens;
    p.block_table = block_table;
    p.free_pages = free_pages;
    p.num_free_in = num_free_in;
    p.num_free_out = num_free_out;
    p.seq_lens = seq_lens;
    p.q_indptr = q_indptr;
    p.kv_indptr = kv_indptr;
    p.slot_mapping = slot_mapping;
    p.positions = positions;
    p.dev_status = dev_status;
    p.batch = batch;
    p.max_pages = max_pages_per_seq;
    p.num_pages = num_pages;
    p.free_capacity = free_capacity;
    p.max_tokens = max_tokens;
    return from_cuda(launch_plan_step(p, to_cuda(stream)));
}

nvfp4kv_status nvfp4kv_release_pages(const int32_t *old_lens, const int32_t *keep_lens, int32_t batch,
                                     const int32_t *block_table, int32_t max_pages_per_seq, int32_t num_pages,
                                     int32_t *free_pages, int32_t free_capacity, const int32_t *num_free_in,
                                     int32_t *num_free_out, int32_t *dev_status, nvfp4kv_stream_t stream)
{
    const nvfp4kv_status st = check_tables(old_lens, keep_lens, batch, block_table, max_pages_per_seq, num_pages,
                                           free_pages, free_capacity, num_free_in, num_free_out);
    if (st != NVFP4KV_OK)
        return st;
    const size_t n = 4 * static_cast<size_t>(batch);
    const Span spans[] = {{old_lens, n, false},
                          {keep_lens, n, false},
                          {block_table, n * static_cast<size_t>(max_pages_per_seq), false},
                          {num_free_in, 4, false},
                          {num_free_out == num_free_in ? nullptr : num_free_out, 4, true},
                          {free_pages, 4 * static_cast<size_t>(free_capacity), true},
                          {dev_status, 4, true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    StepTablesParams p{};
    p.lens_a = old_lens;
    p.lens_b = keep_lens;
    p.block_table = const_cast<int32_t *>(block_table);
    p.free_pages = free_pages;
    p.free_pages_out = free_pages;
    p.num_free_in = num_free_in;
    p.num_free_out = num_free_out;
    p.dev_status = dev_status;
    p.batch = batch;
    p.max_pages = max_pages_per_seq;
    p.num_pages = num_pages;
    p.free_capacity = free_capacity;
    return from_cuda(launch_release_pages(p, to_cuda(stream)));
}

nvfp4kv_status nvfp4kv_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                    nvfp4kv_dtype in_dtype, int32_t num_tokens, int32_t num_q_heads,
                                    int32_t num_kv_heads, const int32_t *positions, const nvfp4kv_rope *rope,
                                    const nvfp4kv_head_norm *norm, void *q_out, void *k_out,
                                    int32_t *dev_status, nvfp4kv_stream_t stream)
{
    NormRopeParams p;
    const nvfp4kv_status st = check_norm_rope(q, q_stride, k, k_stride, in_dtype, num_tokens, num_q_heads,
                                              num_kv_heads, positions, rope, norm, q_out, p);
    if (st != NVFP4KV_OK || num_tokens == 0)
        return st;
    if (k_out == nullptr || !aligned16(k_out))
        return NVFP4KV_ERR_INVALID_ARG;
    const int size = p.in_bf16 ? 2 : 4;
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * kHeadDim;
    const int64_t k_row = static_cast<int64_t>(num_kv_heads) * kHeadDim;
    const bool q_same = q_out == q && p.in_bf16 && q_stride == q_row;    // a row is read whole before it is written
    const bool k_same = k_out == k && k_stride == k_row;
    const size_t t = static_cast<size_t>(num_tokens), norm_bytes = kHeadDim * (p.weight_bf16 ? 2 : 4);
    const Span spans[] = {{q_same ? nullptr : q, rows_bytes(q_stride, num_tokens, num_q_heads, size), false},
                          {k_same ? nullptr : k, rows_bytes(k_stride, num_tokens, num_kv_heads, size), false},
                          {positions, 4 * t, false},
                          {p.q_weight, norm_bytes, false},
                          {p.k_weight, norm_bytes, false},
                          {q_out, t * q_row * 2, true},
                          {k_out, t * k_row * size, true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    p.k_out = k_out;
    p.dev_status = dev_status;
    return from_cuda(launch_norm_rope(p, to_cuda(stream)));
}

nvfp4kv_status nvfp4kv_qk_norm_rope_append(const nvfp4kv_cache *cache, const void *q, int64_t q_stride,
                                           const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                           nvfp4kv_dtype in_dtype, int32_t num_tokens, int32_t num_q_heads,
                                           const int32_t *positions, const int32_t *slot_mapping,
                                           const nvfp4kv_rope *rope, const nvfp4kv_head_norm *norm, void *q_out,
                                           int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_nvfp4(cache);
    if (st != NVFP4KV_OK)
        return st;
    NormRopeParams p;
    st = check_norm_rope(q, q_stride, k, k_stride, in_dtype, num_tokens, num_q_heads, cache->num_kv_heads, positions,
                         rope, norm, q_out, p);
    if (st != NVFP4KV_OK || num_tokens == 0)
        return st;
    if (static_cast<int64_t>(cache->num_pages) * kPageSize > (int64_t{1} << 31) - 1)
        return NVFP4KV_ERR_UNSUPPORTED;      // slots are int32
    const int size = p.in_bf16 ? 2 : 4;
    if (!good_rows(v, v_stride, cache->num_kv_heads, size) || slot_mapping == nullptr || !aligned4(slot_mapping))
        return NVFP4KV_ERR_INVALID_ARG;
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * kHeadDim;
    const bool q_same = q_out == q && p.in_bf16 && q_stride == q_row;
    const size_t t = static_cast<size_t>(num_tokens), norm_bytes = kHeadDim * (p.weight_bf16 ? 2 : 4);
    const Span spans[] = {{q_same ? nullptr : q, rows_bytes(q_stride, num_tokens, num_q_heads, size), false},
                          {k, rows_bytes(k_stride, num_tokens, p.hkv, size), false},
                          {v, rows_bytes(v_stride, num_tokens, p.hkv, size), false},
                          {positions, 4 * t, false},
                          {slot_mapping, 4 * t, false},
                          {p.q_weight, norm_bytes, false},
                          {p.k_weight, norm_bytes, false},
                          {q_out, t * q_row * 2, true},
                          {cache->pool, static_cast<size_t>(cache->num_pages) * p.hkv * kNvfp4Record, true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    p.v = v;
    p.v_stride = v_stride;
    p.slot_mapping = slot_mapping;
    p.pool = static_cast<uint8_t *>(cache->pool);
    p.num_pages = cache->num_pages;
    p.gscale = cache->global_scale;
    p.hs = head_scales_of(cache);
    p.dev_status = dev_status;
    return from_cuda(launch_norm_rope(p, to_cuda(stream)));
}

nvfp4kv_status fp8kv_quantize_append(const fp8kv_cache *cache, const void *k_new, const void *v_new,
                                     nvfp4kv_dtype in_dtype, int32_t num_tokens, const int32_t *slot_mapping,
                                     int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_fp8(cache);
    if (st != NVFP4KV_OK)
        return st;
    st = check_append(k_new, v_new, in_dtype, num_tokens, slot_mapping);
    if (st != NVFP4KV_OK || num_tokens == 0)
        return st;
    QuantParams p{};
    p.k_new = k_new;
    p.v_new = v_new;
    p.slot_mapping = slot_mapping;
    p.pool = static_cast<uint8_t *>(cache->pool);
    p.dev_status = dev_status;
    p.num_tokens = num_tokens;
    p.hkv = cache->num_kv_heads;
    p.num_pages = cache->num_pages;
    p.in_bf16 = in_dtype == NVFP4KV_BF16;
    return from_cuda(launch_quantize_append_fp8(p, to_cuda(stream)));
}

nvfp4kv_status fp8kv_paged_decode(const fp8kv_cache *cache, const void *q, int32_t batch, int32_t num_q_heads,
                                  const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
                                  float sm_scale, void *out, nvfp4kv_dtype out_dtype, void *workspace,
                                  size_t workspace_bytes, int32_t num_workers, int32_t *dev_status,
                                  nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_fp8(cache);
    if (st != NVFP4KV_OK)
        return st;
    DecodeParams p;
    st = check_decode(cache->num_kv_heads, cache->num_pages, q, batch, num_q_heads, block_table,
                      max_pages_per_seq, seq_lens, sm_scale, out, out_dtype, workspace, workspace_bytes,
                      num_workers, dev_status, p);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    p.pool = static_cast<const uint8_t *>(cache->pool);
    cudaError_t e = launch_decode_fp8(p, to_cuda(stream));
    if (e == cudaSuccess)
        e = launch_merge(p, to_cuda(stream));
    return from_cuda(e);
}

nvfp4kv_status nvfp4kv_append_paged_decode(const nvfp4kv_cache *cache, const void *k_new, const void *v_new,
                                           nvfp4kv_dtype in_dtype, const void *q, int32_t batch,
                                           int32_t num_q_heads, const int32_t *block_table,
                                           int32_t max_pages_per_seq, const int32_t *seq_lens, float sm_scale,
                                           void *out, nvfp4kv_dtype out_dtype, void *workspace,
                                           size_t workspace_bytes, int32_t num_workers, int32_t *dev_status,
                                           nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_nvfp4(cache);
    if (st != NVFP4KV_OK)
        return st;
    st = check_append(k_new, v_new, in_dtype, batch, block_table);
    if (st != NVFP4KV_OK)
        return st;
    DecodeParams p;
    st = check_decode(cache->num_kv_heads, cache->num_pages, q, batch, num_q_heads, block_table,
                      max_pages_per_seq, seq_lens, sm_scale, out, out_dtype, workspace, workspace_bytes,
                      num_workers, dev_status, p);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    p.pool = static_cast<const uint8_t *>(cache->pool);
    apply_tensor_scale(p, sm_scale, cache);
    p.k_new = k_new;
    p.v_new = v_new;
    p.append = 1;
    p.new_bf16 = in_dtype == NVFP4KV_BF16;
    cudaError_t e = launch_decode_nvfp4(p, to_cuda(stream));
    if (e == cudaSuccess)
        e = launch_merge(p, to_cuda(stream));
    return from_cuda(e);
}

nvfp4kv_status fp8kv_append_paged_decode(const fp8kv_cache *cache, const void *k_new, const void *v_new,
                                         nvfp4kv_dtype in_dtype, const void *q, int32_t batch,
                                         int32_t num_q_heads, const int32_t *block_table,
                                         int32_t max_pages_per_seq, const int32_t *seq_lens, float sm_scale,
                                         void *out, nvfp4kv_dtype out_dtype, void *workspace,
                                         size_t workspace_bytes, int32_t num_workers, int32_t *dev_status,
                                         nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_fp8(cache);
    if (st != NVFP4KV_OK)
        return st;
    st = check_append(k_new, v_new, in_dtype, batch, block_table);
    if (st != NVFP4KV_OK)
        return st;
    DecodeParams p;
    st = check_decode(cache->num_kv_heads, cache->num_pages, q, batch, num_q_heads, block_table,
                      max_pages_per_seq, seq_lens, sm_scale, out, out_dtype, workspace, workspace_bytes,
                      num_workers, dev_status, p);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    p.pool = static_cast<const uint8_t *>(cache->pool);
    p.k_new = k_new;
    p.v_new = v_new;
    p.append = 1;
    p.new_bf16 = in_dtype == NVFP4KV_BF16;
    cudaError_t e = launch_decode_fp8(p, to_cuda(stream));
    if (e == cudaSuccess)
        e = launch_merge(p, to_cuda(stream));
    return from_cuda(e);
}

nvfp4kv_status fp8bkv_append(const fp8bkv_cache *cache, const void *k_new, const void *v_new, nvfp4kv_dtype in_dtype,
                             int32_t num_tokens, const int32_t *q_indptr, int32_t batch, const int32_t *block_table,
                             int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t *dev_status,
                             nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_fp8(cache);
    if (st != NVFP4KV_OK)
        return st;
    st = check_append(k_new, v_new, in_dtype, num_tokens, q_indptr);
    if (st != NVFP4KV_OK)
        return st;
    st = check_rows(batch, block_table, max_pages_per_seq, seq_lens, nullptr);
    if (st != NVFP4KV_OK || num_tokens == 0 || batch == 0)
        return st;
    const size_t n = 4 * static_cast<size_t>(batch), size = in_dtype == NVFP4KV_BF16 ? 2 : 4;
    const size_t row = static_cast<size_t>(cache->num_kv_heads) * kHeadDim * size;
    const Span spans[] = {{k_new, num_tokens * row, false},
                          {v_new, num_tokens * row, false},
                          {q_indptr, n + 4, false},
                          {block_table, n * static_cast<size_t>(max_pages_per_seq), false},
                          {seq_lens, n, false},
                          {cache->pool, static_cast<size_t>(cache->num_pages) * cache->num_kv_heads * kFp8BlockRecord, true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    BlockAppendParams p{};
    p.k_new = k_new;
    p.v_new = v_new;
    p.q_indptr = q_indptr;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.pool = static_cast<uint8_t *>(cache->pool);
    p.dev_status = dev_status;
    p.num_tokens = num_tokens;
    p.batch = batch;
    p.hkv = cache->num_kv_heads;
    p.max_pages = max_pages_per_seq;
    p.num_pages = cache->num_pages;
    p.in_bf16 = in_dtype == NVFP4KV_BF16;
    return from_cuda(launch_block_append(p, to_cuda(stream)));
}

nvfp4kv_status fp8bkv_dequant(const fp8bkv_cache *cache, const int32_t *block_table, int32_t max_pages_per_seq,
                              const int32_t *lens, const int32_t *kv_indptr, int32_t batch, void *k_out, void *v_out,
                              nvfp4kv_dtype out_dtype, int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_fp8(cache);
    if (st != NVFP4KV_OK)
        return st;
    if (out_dtype != NVFP4KV_F32 && out_dtype != NVFP4KV_BF16 && out_dtype != NVFP4KV_E4M3)
        return NVFP4KV_ERR_INVALID_ARG;
    st = check_rows(batch, block_table, max_pages_per_seq, lens, kv_indptr);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    if (kv_indptr == nullptr || k_out == nullptr || v_out == nullptr || !aligned16(k_out) || !aligned16(v_out))
        return NVFP4KV_ERR_INVALID_ARG;
    // (how many rows the outputs have, only the device knows: one each is looked at)
    const size_t n = 4 * static_cast<size_t>(batch);
    const size_t row = static_cast<size_t>(cache->num_kv_heads) * kHeadDim *
                       (out_dtype == NVFP4KV_F32 ? 4 : (out_dtype == NVFP4KV_BF16 ? 2 : 1));
    const Span spans[] = {{cache->pool, static_cast<size_t>(cache->num_pages) * cache->num_kv_heads * kFp8BlockRecord, false},
                          {block_table, n * static_cast<size_t>(max_pages_per_seq), false},
                          {lens, n, false},
                          {kv_indptr, n, false},
                          {k_out, row, true},
                          {v_out, row, true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    BlockReadParams p{};
    p.pool = static_cast<const uint8_t *>(cache->pool);
    p.block_table = block_table;
    p.lens = lens;
    p.kv_indptr = kv_indptr;
    p.k_out = k_out;
    p.v_out = v_out;
    p.dev_status = dev_status;
    p.batch = batch;
    p.hkv = cache->num_kv_heads;
    p.max_pages = max_pages_per_seq;
    p.num_pages = cache->num_pages;
    p.out_dtype = out_dtype;
    return from_cuda(launch_block_read(p, to_cuda(stream)));
}

nvfp4kv_status fp8bkv_paged_decode(const fp8bkv_cache *cache, const void *q, int32_t batch, int32_t q_len,
                                   int32_t num_q_heads, const int32_t *block_table, int32_t max_pages_per_seq,
                                   const int32_t *seq_lens, float sm_scale, void *out, nvfp4kv_dtype out_dtype,
                                   void *workspace, size_t workspace_bytes, int32_t num_workers, int32_t *dev_status,
                                   nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_fp8(cache);
    if (st != NVFP4KV_OK)
        return st;
    if (q_len < 1 || q_len > NVFP4KV_MAX_QUERY_TOKENS)
        return q_len < 1 ? NVFP4KV_ERR_INVALID_ARG : NVFP4KV_ERR_UNSUPPORTED;
    DecodeParams p;
    st = check_decode(cache->num_kv_heads, cache->num_pages, q, batch, num_q_heads, block_table, max_pages_per_seq,
                      seq_lens, sm_scale, out, out_dtype, workspace, workspace_bytes, num_workers, dev_status, p);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    const size_t elems = static_cast<size_t>(batch) * q_len * num_q_heads * kHeadDim;
    const Span spans[] = {{q, 2 * elems, false},
                          {block_table, 4 * static_cast<size_t>(batch) * max_pages_per_seq, false},
                          {seq_lens, 4 * static_cast<size_t>(batch), false},
                          {cache->pool, static_cast<size_t>(cache->num_pages) * cache->num_kv_heads * kFp8BlockRecord, false},
                          {out, elems * (out_dtype == NVFP4KV_F32 ? 4 : 2), true},
                          {workspace, decode_workspace_bytes(p.num_workers), true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    p.pool = static_cast<const uint8_t *>(cache->pool);
    const int rows = p.group * q_len, row_groups = (rows + kMaxGroup - 1) / kMaxGroup;
    const int64_t heads = static_cast<int64_t>(batch) * p.hkv;
    // short sequences: each query token by a cluster of its own
    const ClusterPlan plan = num_workers == 0 ? plan_cluster_decode(heads * q_len, heads * row_groups, max_pages_per_seq,
                                                                    true, false, q_len)
                                              : ClusterPlan{};
    if (plan.first > 0) {
        p.batch = batch * q_len;
        p.sel_q_len = q_len;
        return from_cuda(launch_cluster_decode_fp8_block(p, plan, to_cuda(stream)));
    }
    p.q_len = q_len;
    p.rows = rows;
    p.row_groups = row_groups;
    if (static_cast<int64_t>(batch) * cache->num_kv_heads * p.row_groups * max_pages_per_seq > (int64_t{1} << 31) - 1)
        return NVFP4KV_ERR_UNSUPPORTED;
    p.lanes = p.row_groups > 1 && p.num_workers >= p.row_groups ? p.row_groups : 1;
    cudaError_t e = launch_decode_fp8_block(p, to_cuda(stream));
    if (e == cudaSuccess)
        e = launch_merge(p, to_cuda(stream));
    return from_cuda(e);
}

nvfp4kv_status nvfp4kv_page_bounds(const nvfp4kv_cache *cache, const nvfp4kv_bounds *bounds,
                                   const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *from_lens,
                                   const int32_t *seq_lens, int32_t batch, int32_t *dev_status,
                                   nvfp4kv_stream_t stream)
{
    const nvfp4kv_status st = check_nvfp4(cache);
    if (st != NVFP4KV_OK)
        return st;
    return page_bounds(cache, kNvfp4Record, bounds, block_table, max_pages_per_seq, from_lens, seq_lens, batch,
                       dev_status, stream, launch_page_bounds_nvfp4);
}

nvfp4kv_status fp8bkv_page_bounds(const fp8bkv_cache *cache, const nvfp4kv_bounds *bounds, const int32_t *block_table,
                                  int32_t max_pages_per_seq, const int32_t *from_lens, const int32_t *seq_lens,
                                  int32_t batch, int32_t *dev_status, nvfp4kv_stream_t stream)
{
    const nvfp4kv_status st = check_fp8(cache);
    if (st != NVFP4KV_OK)
        return st;
    return page_bounds(cache, kFp8BlockRecord, bounds, block_table, max_pages_per_seq, from_lens, seq_lens, batch,
                       dev_status, stream, launch_page_bounds_fp8_block);
}

nvfp4kv_status nvfp4kv_select_pages(const nvfp4kv_bounds *bounds, const void *q, int32_t batch, int32_t q_len,
                                    int32_t num_q_heads, const int32_t *block_table, int32_t max_pages_per_seq,
                                    const int32_t *seq_lens, int32_t budget, int32_t first_pages, int32_t last_pages,
                                    int32_t *pages, int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_bounds(bounds);
    if (st != NVFP4KV_OK)
        return st;
    const int32_t hkv = bounds->num_kv_heads;
    st = check_select_sizes(batch, q_len, hkv, max_pages_per_seq);
    if (st == NVFP4KV_OK)
        st = check_rows(batch, block_table, max_pages_per_seq, seq_lens, pages);
    if (st != NVFP4KV_OK)
        return st;
    if (num_q_heads <= 0 || num_q_heads % hkv != 0 || budget <= 0 || first_pages < 0 || last_pages < 0 ||
        first_pages > budget - last_pages)
        return NVFP4KV_ERR_INVALID_ARG;
    if (num_q_heads / hkv > kMaxGroup)
        return NVFP4KV_ERR_UNSUPPORTED;
    if (batch == 0)
        return NVFP4KV_OK;
    if (q == nullptr || !aligned16(q) || pages == nullptr)
        return NVFP4KV_ERR_INVALID_ARG;
    const size_t rows = static_cast<size_t>(batch) * q_len, heads = heads_of(bounds);
    const Span spans[] = {{bounds->bounds, heads * 2 * kHeadDim, false},
                          {bounds->steps, 4 * heads, false},
                          {q, 2 * rows * num_q_heads * kHeadDim, false},
                          {block_table, 4 * static_cast<size_t>(batch) * max_pages_per_seq, false},
                          {seq_lens, 4 * static_cast<size_t>(batch), false},
                          {pages, 4 * rows * hkv * static_cast<size_t>(budget), true}};
    if (written_overlap(spans))
        return NVFP4KV_ERR_INVALID_ARG;
    SelectParams p{};
    p.bounds = bounds->bounds;
    p.steps = bounds->steps;
    p.q = static_cast<const uint16_t *>(q);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.pages = pages;
    p.dev_status = dev_status;
    p.batch = batch;
    p.q_len = q_len;
    p.hq = num_q_heads;
    p.hkv = hkv;
    p.group = num_q_heads / hkv;
    p.max_pages = max_pages_per_seq;
    p.num_pages = bounds->num_pages;
    p.budget = budget;
    p.first = first_pages;
    p.last = last_pages;
    return from_cuda(launch_select_pages(p, to_cuda(stream)));
}

nvfp4kv_status nvfp4kv_selected_decode(const nvfp4kv_cache *cache, const void *q, int32_t batch, int32_t q_len,
                                       int32_t num_q_heads, const int32_t *block_table, int32_t max_pages_per_seq,
                                       const int32_t *seq_lens, const int32_t *pages, int32_t budget, float sm_scale,
                                       void *out, nvfp4kv_dtype out_dtype, void *workspace, size_t workspace_bytes,
                                       int32_t num_workers, int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_nvfp4(cache);
    if (st != NVFP4KV_OK)
        return st;
    DecodeParams p;
    st = check_selected(cache->num_kv_heads, cache->num_pages,
                        static_cast<size_t>(cache->num_pages) * cache->num_kv_heads * kNvfp4Record, cache->pool, q, batch,
                        q_len, num_q_heads, block_table, max_pages_per_seq, seq_lens, pages, budget, sm_scale, out,
                        out_dtype, workspace, workspace_bytes, num_workers, dev_status, p);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    p.pool = static_cast<const uint8_t *>(cache->pool);
    apply_tensor_scale(p, sm_scale, cache);
    const ClusterPlan plan = num_workers == 0 ? cluster_plan(p, false) : ClusterPlan{};
    if (plan.first > 0)
        return from_cuda(launch_cluster_decode_nvfp4(p, plan, to_cuda(stream)));
    cudaError_t e = launch_decode_selected_nvfp4(p, to_cuda(stream));
    if (e == cudaSuccess)
        e = launch_merge(p, to_cuda(stream));
    return from_cuda(e);
}

nvfp4kv_status fp8bkv_selected_decode(const fp8bkv_cache *cache, const void *q, int32_t batch, int32_t q_len,
                                      int32_t num_q_heads, const int32_t *block_table, int32_t max_pages_per_seq,
                                      const int32_t *seq_lens, const int32_t *pages, int32_t budget, float sm_scale,
                                      void *out, nvfp4kv_dtype out_dtype, void *workspace, size_t workspace_bytes,
                                      int32_t num_workers, int32_t *dev_status, nvfp4kv_stream_t stream)
{
    nvfp4kv_status st = check_fp8(cache);
    if (st != NVFP4KV_OK)
        return st;
    DecodeParams p;
    st = check_selected(cache->num_kv_heads, cache->num_pages,
                        static_cast<size_t>(cache->num_pages) * cache->num_kv_heads * kFp8BlockRecord, cache->pool, q,
                        batch, q_len, num_q_heads, block_table, max_pages_per_seq, seq_lens, pages, budget, sm_scale, out,
                        out_dtype, workspace, workspace_bytes, num_workers, dev_status, p);
    if (st != NVFP4KV_OK || batch == 0)
        return st;
    p.pool = static_cast<const uint8_t *>(cache->pool);
    const ClusterPlan plan = num_workers == 0 ? cluster_plan(p, true) : ClusterPlan{};
    if (plan.first > 0)
        return from_cuda(launch_cluster_decode_fp8_block(p, plan, to_cuda(stream)));
    cudaError_t e = launch_decode_selected_fp8_block(p, to_cuda(stream));
    if (e == cudaSuccess)
        e = launch_merge(p, to_cuda(stream));
    return from_cuda(e);
}

int64_t fp8bkv_cache_bytes(int32_t num_pages, int32_t num_kv_heads, int32_t page_size, int32_t head_dim)
{
    if (num_pages < 0 || num_kv_heads < 0 || page_size != kPageSize || head_dim != kHeadDim)
        return -1;
    return static_cast<int64_t>(num_pages) * num_kv_heads * kFp8BlockRecord;
}

int64_t nvfp4kv_cache_bytes(int32_t num_pages, int32_t num_kv_heads, int32_t page_size, int32_t head_dim)
{
    if (num_pages < 0 || num_kv_heads < 0 || page_size < 0 || head_dim < 0 || head_dim % 16 != 0)
        return -1;
    const int64_t rows = static_cast<int64_t>(num_pages) * num_kv_heads * page_size;
    return 2 * rows * (head_dim / 2 + head_dim / 16);
}

int64_t fp8kv_cache_bytes(int32_t num_pages, int32_t num_kv_heads, int32_t page_size, int32_t head_dim)
{
    if (num_pages < 0 || num_kv_heads < 0 || page_size < 0 || head_dim < 0)
        return -1;
    return 2 * static_cast<int64_t>(num_pages) * num_kv_heads * page_size * head_dim;
}

nvfp4kv_status nvfp4kv_read_device_status(const int32_t *dev_status, nvfp4kv_stream_t stream, int32_t *bits)
{
    if (dev_status == nullptr || bits == nullptr)
        return NVFP4KV_ERR_INVALID_ARG;
    if (cudaStreamSynchronize(to_cuda(stream)) != cudaSuccess)
        return NVFP4KV_ERR_CUDA;
    int32_t v = 0;
    if (cudaMemcpy(&v, dev_status, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess)
        return NVFP4KV_ERR_CUDA;
    *bits = v;
    return v != 0 ? NVFP4KV_ERR_DEVICE_CHECK : NVFP4KV_OK;
}

uint32_t nvfp4kv_set_wait_limit(uint32_t polls)
{
    return g_wait_limit.exchange(polls, std::memory_order_relaxed);
}

const char *nvfp4kv_status_string(nvfp4kv_status status)
{
    switch (status) {
    case NVFP4KV_OK:
        return "ok";
    case NVFP4KV_ERR_INVALID_ARG:
        return "invalid argument";
    case NVFP4KV_ERR_UNSUPPORTED:
        return "unsupported geometry or option";
    case NVFP4KV_ERR_WORKSPACE:
        return "decode workspace missing, misaligned or too small";
    case NVFP4KV_ERR_CUDA:
        return "CUDA runtime error";
    case NVFP4KV_ERR_DEVICE_CHECK:
        return "a kernel reported bad device data (see the status bits)";
    }
    return "unknown status";
}

int32_t nvfp4kv_version(void)
{
    return 100;
}

} // extern "C"
