// A serving step's tables on the GPU: page allocation, block tables, slot and
// position maps from request lengths, and the return of pages.
//
// Request b holds ceil(context_lens[b] / 16) pages and adds new_lens[b]
// tokens; with had = ceil(ctx / 16) and has = ceil((ctx + new) / 16) it takes
// the pages had .. has - 1 from the top of a stack of free page ids.  Fresh
// pages are numbered in the order of (request, page), so fresh page i of the
// step is free_pages[num_free - 1 - i] whatever the launch shape.  Everything
// follows from two exclusive sums over the requests (fresh pages, new tokens)
// and a third of the contexts (the prefix workspace offsets).
//
// The work is a few integers a token, so the time is launch latency and one
// dependent chain: lengths -> sums -> page id -> slot.  Every CTA takes the
// sums over all requests by itself (at most 8,192 pairs of lengths, L2 hits
// for all CTAs but the first) and then fills its share of the token rows and
// of the fresh table entries, finding an item's request by binary search in
// shared memory: one launch, nothing passes between CTAs.  A slot in a fresh
// page takes the page id from the stack, not from the table entry that some
// other CTA writes in the same launch.
#include "device_common.cuh"

namespace nvfp4kv {
namespace {

constexpr int kTablesThreads = 512;
constexpr int kTablesWarps = kTablesThreads / 32;
constexpr int kItemsPerThread = 4;       // token rows a thread fills before another CTA is worth its scan

struct Lens {
    int first, second;                   // pages held before and after, whichever way the call goes
    int a, b;                            // the checked lengths
};

// Lengths a (context, or old) and b (new, or keep) of one request: `bad` when
// they do not describe a request; it then has no tokens and moves no pages.
template <bool kRelease>
__device__ __forceinline__ Lens read_lens(const StepTablesParams &p, int i, bool &bad)
{
    const int max_len = p.max_pages * kPageSize;
    int a = __ldcg(p.lens_a + i), b = __ldcg(p.lens_b + i);
    bad = a < 0 || b < 0 || a > max_len || (kRelease ? b > a : b > max_len - a);
    if (bad)
        a = b = 0;
    const int after = kRelease ? b : a + b;
    return {(a + kPageSize - 1) / kPageSize, (after + kPageSize - 1) / kPageSize, a, b};
}

struct Totals {
    long long pages, tokens, context;
    int num_free;
    bool ok;                             // the step can be taken as a whole
};

// Exclusive sums over the requests into page_at / token_at (batch + 1 entries
// each) and, when kv_indptr is wanted, the context sums; whole CTA.  `rep`:
// this CTA reports what is wrong.  Sums are taken in 64 bits: lengths of up to
// 2^30 over 8,192 requests pass 32; the entries kept are used only when the
// totals fit.
template <bool kRelease>
__device__ __forceinline__ Totals scan_requests(const StepTablesParams &p, int32_t *page_at, int32_t *token_at,
                                                int32_t *kv_indptr, bool rep)
{
    __shared__ long long part[2][kTablesWarps][3];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long carry[3] = {0, 0, 0};
    int turn = 0;
    for (int base = 0; base < p.batch; base += kTablesThreads, turn ^= 1) {
        const int i = base + threadIdx.x;
        long long own[3] = {0, 0, 0};
        if (i < p.batch) {
            bool bad;
            const Lens l = read_lens<kRelease>(p, i, bad);
            if (bad && rep)
                report(p.dev_status, NVFP4KV_DEV_BAD_LEN);
            own[0] = kRelease ? l.first - l.second : l.second - l.first;
            own[1] = kRelease ? 0 : l.b;
            own[2] = kRelease ? 0 : l.a;
        }
        long long incl[3];
#pragma unroll
        for (int k = 0; k < (kRelease ? 1 : 3); ++k) {
            long long x = own[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(kFullMask, x, o);
                if (lane >= o)
                    x += y;
            }
            incl[k] = x;
            if (lane == 31)
                part[turn][warp][k] = x;
        }
        // two buffers in turn: the next round's writes cannot meet this
        // round's reads, which every thread finishes before its next barrier
        __syncthreads();
#pragma unroll
        for (int k = 0; k < (kRelease ? 1 : 3); ++k) {
            long long before = 0, total = 0;
#pragma unroll
            for (int w = 0; w < kTablesWarps; ++w) {
                const long long s = part[turn][w][k];
                before += w < warp ? s : 0;
                total += s;
            }
            const long long at = carry[k] + before + incl[k] - own[k];
            if (i < p.batch) {
                if (k == 0)
                    page_at[i] = static_cast<int32_t>(at);
                else if (k == 1)
                    token_at[i] = static_cast<int32_t>(at);
                else if (kv_indptr != nullptr)
                    kv_indptr[i] = static_cast<int32_t>(at);
            }
            carry[k] += total;
        }
    }
    Totals t{carry[0], carry[1], carry[2], __ldcg(p.num_free_in), true};
    if (t.num_free < 0 || t.num_free > p.free_capacity) {
        if (rep && threadIdx.x == 0)
            report(p.dev_status, NVFP4KV_DEV_BAD_LEN);
        t.num_free = t.num_free < 0 ? 0 : p.free_capacity;
        t.ok = false;
    }
    if (kRelease) {
        if (t.ok && t.pages > p.free_capacity - t.num_free) {
            t.ok = false;
            if (rep && threadIdx.x == 0)
                report(p.dev_status, NVFP4KV_DEV_BAD_LEN);
        }
    } else {
        if (t.ok && t.pages > t.num_free) {
            t.ok = false;
            if (rep && threadIdx.x == 0)
                report(p.dev_status, NVFP4KV_DEV_NO_PAGES);
        }
        if (t.tokens > p.max_tokens || t.context > 0x7fffffffLL) {
            t.ok = false;
            if (rep && threadIdx.x == 0)
                report(p.dev_status, NVFP4KV_DEV_BAD_LEN);
        }
    }
    if (threadIdx.x == 0) {
        page_at[p.batch] = static_cast<int32_t>(t.pages);
        if (!kRelease)
            token_at[p.batch] = static_cast<int32_t>(t.tokens);
    }
    __syncthreads();
    return t;
}

// Largest i with at[i] <= x (the request that holds item x, 0 <= x < at[n]).
__device__ __forceinline__ int find_request(const int32_t *at, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Lengths, the old table entries and the stack are read past the first-level
// cache (ld.cg): the next step's kernels may read the same lines on this SM.
__global__ void __launch_bounds__(kTablesThreads) plan_step_kernel(const __grid_constant__ StepTablesParams p)
{
    extern __shared__ int32_t smem_at[];
    int32_t *page_at = smem_at, *token_at = smem_at + p.batch + 1;
    const bool head = blockIdx.x == 0;
    const Totals t = scan_requests<false>(p, page_at, token_at, head ? p.kv_indptr : nullptr, head);
    const int stride = static_cast<int>(gridDim.x) * kTablesThreads;
    const int first = static_cast<int>(blockIdx.x) * kTablesThreads + threadIdx.x;

    for (int i = first; i <= p.batch; i += stride) {
        p.q_indptr[i] = t.ok ? token_at[i] : 0;
        if (i < p.batch) {
            bool bad;
            const Lens l = read_lens<false>(p, i, bad);
            p.seq_lens[i] = l.a + (t.ok ? l.b : 0);
        }
    }
    if (head && p.kv_indptr != nullptr && t.context > 0x7fffffffLL) {
        // offsets that would pass 32 bits: none
        for (int i = threadIdx.x; i < p.batch; i += kTablesThreads)
            p.kv_indptr[i] = 0;
    }
    const int tokens = t.ok ? static_cast<int>(t.tokens) : 0;
    const int pages = t.ok ? static_cast<int>(t.pages) : 0;
    for (int i = first; i < pages; i += stride) {
        const int b = find_request(page_at, p.batch, i);
        bool bad;
        const Lens l = read_lens<false>(p, b, bad);
        const int j = l.first + (i - page_at[b]);
        p.block_table[static_cast<size_t>(b) * p.max_pages + j] = __ldcg(p.free_pages + (t.num_free - 1 - i));
    }
    for (long long r = first; r < p.max_tokens; r += stride) {
        int pos = -1, slot = -1;
        if (r < tokens) {
            const int b = find_request(token_at, p.batch, static_cast<int>(r));
            bool bad;
            const Lens l = read_lens<false>(p, b, bad);
            pos = l.a + (static_cast<int>(r) - token_at[b]);
            const int j = pos / kPageSize;
            const int page = j >= l.first
                                 ? __ldcg(p.free_pages + (t.num_free - 1 - (page_at[b] + j - l.first)))
                                 : __ldcg(p.block_table + static_cast<size_t>(b) * p.max_pages + j);
            if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages))
                slot = page * kPageSize + pos % kPageSize;
            else
                report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);
        }
        p.slot_mapping[r] = slot;
        if (p.positions != nullptr)
            p.positions[r] = pos;
    }
    // (one CTA: every thread has read num_free_in before the scan's last barrier)
    if (p.count_here && head && threadIdx.x == 0)
        *p.num_free_out = t.num_free - pages;
    __threadfence();
}

// Pages ceil(keep / 16) .. ceil(old / 16) - 1 of every request go back on the
// stack in the order of (request, page).
__global__ void __launch_bounds__(kTablesThreads) release_pages_kernel(const __grid_constant__ StepTablesParams p)
{
    extern __shared__ int32_t smem_at[];
    int32_t *page_at = smem_at;
    const bool head = blockIdx.x == 0;
    const Totals t = scan_requests<true>(p, page_at, nullptr, nullptr, head);
    const int pages = t.ok ? static_cast<int>(t.pages) : 0;
    const int stride = static_cast<int>(gridDim.x) * kTablesThreads;
    for (long long i = static_cast<long long>(blockIdx.x) * kTablesThreads + threadIdx.x; i < pages; i += stride) {
        const int b = find_request(page_at, p.batch, static_cast<int>(i));
        bool bad;
        const Lens l = read_lens<true>(p, b, bad);
        const int page = __ldcg(p.block_table + static_cast<size_t>(b) * p.max_pages + l.second +
                                (static_cast<int>(i) - page_at[b]));
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages))
            report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);
        p.free_pages_out[t.num_free + i] = page;
    }
    if (p.count_here && head && threadIdx.x == 0)
        *p.num_free_out = t.num_free + pages;
    __threadfence();
}

// The new count when it replaces the one that every CTA of the launch before
// has to read: one CTA, after that launch.
template <bool kRelease>
__global__ void __launch_bounds__(kTablesThreads) free_count_kernel(const __grid_constant__ StepTablesParams p)
{
    extern __shared__ int32_t smem_at[];
    const Totals t = scan_requests<kRelease>(p, smem_at, smem_at + p.batch + 1, nullptr, false);
    if (threadIdx.x == 0) {
        const int pages = t.ok ? static_cast<int>(t.pages) : 0;
        *p.num_free_out = kRelease ? t.num_free + pages : t.num_free - pages;
    }
}

template <class K>
cudaError_t launch_tables(K kernel, K count, StepTablesParams p, long long items, cudaStream_t s)
{
    const long long want = (items + kItemsPerThread * kTablesThreads - 1) / (kItemsPerThread * kTablesThreads);
    const int grid = static_cast<int>(want < 1 ? 1 : (want > sm_count() ? sm_count() : want));
    const size_t smem = 2 * (static_cast<size_t>(p.batch) + 1) * sizeof(int32_t);
    p.count_here = grid == 1 || p.num_free_in != p.num_free_out;
    if (smem > 48 * 1024)
        for (K k : {kernel, count}) {
            // (what the largest batch takes, for other threads' launches too)
            const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       2 * (kMaxBatch + 1) * static_cast<int>(sizeof(int32_t)));
            if (e != cudaSuccess)
                return e;
        }
    kernel<<<grid, kTablesThreads, smem, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.count_here)
        return e;
    count<<<1, kTablesThreads, smem, s>>>(p);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_plan_step(const StepTablesParams &p, cudaStream_t s)
{
    return launch_tables(plan_step_kernel, free_count_kernel<false>, p, p.max_tokens, s);
}

cudaError_t launch_release_pages(const StepTablesParams &p, cudaStream_t s)
{
    return launch_tables(release_pages_kernel, free_count_kernel<true>, p,
                         static_cast<long long>(p.batch) * p.max_pages, s);
}

} // namespace nvfp4kv
