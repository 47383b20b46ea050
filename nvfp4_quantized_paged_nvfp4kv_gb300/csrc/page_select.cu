// Which pages a query looks at: bounds of each page's keys, a score of each page
// from them, and the selection of the best.
//
// Bounds of a page-head over its cached tokens, before the tensor scale: u the
// largest |k|, r = fl32(127 / u), and for each channel c
//   hi_c = min(127, ceil(fl32(max_t k_tc * r))), lo_c = max(-127, floor(fl32(min_t k_tc * r))),
// in steps of fl32(u / 127) (u = 0: all zero), one byte each.
// Queries of a kv head's group, in whole steps too: w = rint(fl32(q * fl32(127 / max |q|))),
// the maximum over the group.  The score of a page is what its best key could
// reach with the best head,
//   score = fl32(step * max_h I_h),  I_h = sum_c (w_hc > 0 ? w_hc hi_c : w_hc lo_c).
// I is a whole number of at most 128 * 127^2 < 2^24, exact in any order of sums,
// and the product is one rounding: the selection is the same whatever the work
// split.  Positive and negative parts of w make I a product of 256 terms,
// (w+, w-) . (hi, lo), which runs on the tensor cores in 8-bit integers.
// A query takes the first pages and the last ones of its sequence and, of the
// others, those of the largest scores, the lower page first where they tie.
#include "decode_common.cuh"

namespace nvfp4kv {
namespace {

// ---- bounds --------------------------------------------------------------------

constexpr int kBoundThreads = 256;

__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Keys of a page-head by lane: kRegs f16x2 (channel pairs from first(lane) on) of
// kTokens tokens.  The lanes that share channels differ in the bits kShare of the
// lane; value(x) = x * scale is exact in fp32.
struct Nvfp4Keys {
    static constexpr int kRecord = kNvfp4Record, kRegs = 16, kTokens = 2, kTopBit = 16, kLowBit = 4;
    uint4 d[2];
    uint32_t s[2];

    __device__ __forceinline__ void load(const uint8_t *rec, int lane)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            d[i] = __ldg(reinterpret_cast<const uint4 *>(rec) + 32 * i + lane);
            s[i] = __ldg(reinterpret_cast<const uint16_t *>(rec + 2048) + 32 * i + lane);
        }
    }
    __device__ __forceinline__ float scale() const { return 1.f; }
    __device__ static __forceinline__ int token(int i, int lane) { return 8 * i + (lane >> 2); }
    __device__ static __forceinline__ int first(int lane) { return 32 * (lane & 3); }
    __device__ __forceinline__ void get(int i, uint32_t (&x)[16]) const
    {
        const uint32_t w[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
        const uint32_t sc = e4m3x2_to_f16x2(s[i]);
        const uint32_t s0 = __byte_perm(sc, 0, 0x1010), s1 = __byte_perm(sc, 0, 0x3232);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            e2m1x8_to_f16x2x4(w[k], x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
#pragma unroll
        for (int k = 0; k < 16; ++k)
            x[k] = hmul2(x[k], k < 8 ? s0 : s1);
    }
};

struct Fp8BlockKeys {
    static constexpr int kRecord = kFp8BlockRecord, kRegs = 8, kTokens = 4, kTopBit = 16, kLowBit = 8;
    uint4 d[4];
    float s;

    __device__ __forceinline__ void load(const uint8_t *rec, int lane)
    {
        const int place = ((lane & 7) + ((lane >> 3) & 1)) & 7;      // of chunk lane % 8 in rows of this parity
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] = __ldg(reinterpret_cast<const uint4 *>(rec) + 32 * i + (lane & ~7) + place);
        s = __ldg(reinterpret_cast<const float *>(rec + kFp8Record));
    }
    __device__ __forceinline__ float scale() const { return s; }
    __device__ static __forceinline__ int token(int i, int lane) { return 4 * i + (lane >> 3); }
    __device__ static __forceinline__ int first(int lane) { return 16 * (lane & 7); }
    __device__ __forceinline__ void get(int i, uint32_t (&x)[8]) const
    {
        const uint32_t w[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            e4m3x4_to_f16x2x2(w[k], x[2 * k], x[2 * k + 1]);
    }
};

// Combine lo / hi over the lanes that share channels, halving what a lane keeps
// with each exchange: in the end two registers, four channels.  Returns the
// first of them (relative to the lane's).
template <int kRegs, int kBit, int kLowBit>
__device__ __forceinline__ int gather_bounds(uint32_t (&lo)[kRegs], uint32_t (&hi)[kRegs], int lane, uint32_t (&out)[4])
{
    constexpr int kHalf = kRegs / 2;
    const bool upper = lane & kBit;
    uint32_t l2[kHalf], h2[kHalf];
#pragma unroll
    for (int k = 0; k < kHalf; ++k) {
        const uint32_t lo_away = upper ? lo[k] : lo[k + kHalf], hi_away = upper ? hi[k] : hi[k + kHalf];
        const uint32_t lo_keep = upper ? lo[k + kHalf] : lo[k], hi_keep = upper ? hi[k + kHalf] : hi[k];
        l2[k] = hmin2(lo_keep, __shfl_xor_sync(kFullMask, lo_away, kBit));
        h2[k] = hmax2(hi_keep, __shfl_xor_sync(kFullMask, hi_away, kBit));
    }
    const int at = upper ? 2 * kHalf : 0;
    if constexpr (kBit == kLowBit) {
        static_assert(kHalf == 2, "four channels a lane");
        out[0] = l2[0];
        out[1] = l2[1];
        out[2] = h2[0];
        out[3] = h2[1];
        return at;
    } else {
        return at + gather_bounds<kHalf, kBit / 2, kLowBit>(l2, h2, lane, out);
    }
}

// One warp a (page, kv head).
template <class Keys>
__global__ void __launch_bounds__(kBoundThreads) page_bounds_kernel(const __grid_constant__ BoundsParams p)
{
    extern __shared__ int32_t bsmem[];
    int32_t *scratch = bsmem, *prefix = bsmem + kPrefixScratch;
    pdl_wait();
    pdl_launch_dependents();
    const int max_len = p.max_pages * kPageSize;
    auto first_page = [&](int b, int len) {
        const int from = p.from_lens == nullptr ? 0 : __ldg(p.from_lens + b);
        return from < len ? max(from, 0) / kPageSize : (len + kPageSize - 1) / kPageSize;
    };
    build_prefix_of(
        [&](int b) {
            const int from = p.from_lens == nullptr ? 0 : __ldg(p.from_lens + b), len = __ldg(p.seq_lens + b);
            if (blockIdx.x == 0 && (len < 0 || len > max_len || from < 0))
                report(p.dev_status, NVFP4KV_DEV_BAD_LEN);
            const int n = clamp_len(len, max_len);
            return (n + kPageSize - 1) / kPageSize - first_page(b, n);
        },
        p.batch, prefix, scratch);
    const int lane = threadIdx.x & 31;
    const long long units = static_cast<long long>(prefix[p.batch]) * p.hkv;
    const long long step = static_cast<long long>(gridDim.x) * (kBoundThreads / 32);
    for (long long u = static_cast<long long>(blockIdx.x) * (kBoundThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
        const int pg = static_cast<int>(u / p.hkv), h = static_cast<int>(u - static_cast<long long>(pg) * p.hkv);
        const int b = find_seq(prefix, p.batch, pg);
        const int len = clamp_len(__ldg(p.seq_lens + b), max_len);
        const int page = first_page(b, len) + pg - prefix[b];
        const int phys = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + page);
        if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_pages)) {
            if (h == 0 && lane == 0)
                report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);
            continue;
        }
        const size_t head = static_cast<size_t>(phys) * p.hkv + h;
        Keys keys;
        keys.load(p.pool + head * Keys::kRecord, lane);
        uint32_t lo[Keys::kRegs], hi[Keys::kRegs];
#pragma unroll
        for (int k = 0; k < Keys::kRegs; ++k) {
            lo[k] = 0x7c007c00u;                             // +inf, -inf
            hi[k] = 0xfc00fc00u;
        }
        const int valid = len - page * kPageSize;
#pragma unroll
        for (int i = 0; i < Keys::kTokens; ++i) {
            if (Keys::token(i, lane) >= valid)
                continue;
            uint32_t x[Keys::kRegs];
            keys.get(i, x);
#pragma unroll
            for (int k = 0; k < Keys::kRegs; ++k) {
                lo[k] = hmin2(lo[k], x[k]);
                hi[k] = hmax2(hi[k], x[k]);
            }
        }
        uint32_t four[4];
        const int c = Keys::first(lane) + gather_bounds<Keys::kRegs, Keys::kTopBit, Keys::kLowBit>(lo, hi, lane, four);
        float l[4], g[4], top = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&four[k]));
            const float2 d = __half22float2(*reinterpret_cast<__half2 *>(&four[2 + k]));
            l[2 * k] = a.x * keys.scale();
            l[2 * k + 1] = a.y * keys.scale();
            g[2 * k] = d.x * keys.scale();
            g[2 * k + 1] = d.y * keys.scale();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            top = fmaxf(top, fmaxf(fabsf(l[k]), fabsf(g[k])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
        const float r = top > 0.f ? __fdiv_rn(127.f, top) : 0.f;
        uint32_t wl = 0, wg = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int a = static_cast<int>(fmaxf(floorf(__fmul_rn(l[k], r)), -127.f));
            const int d = static_cast<int>(fminf(ceilf(__fmul_rn(g[k], r)), 127.f));
            wl |= (static_cast<uint32_t>(a) & 0xffu) << (8 * k);
            wg |= (static_cast<uint32_t>(d) & 0xffu) << (8 * k);
        }
        int8_t *dst = p.bounds + head * (2 * kHeadDim) + c;
        *reinterpret_cast<uint32_t *>(dst) = wl;
        *reinterpret_cast<uint32_t *>(dst + kHeadDim) = wg;
        if (lane == 0)
            p.steps[head] = __fdiv_rn(top, 127.f);
    }
}

template <class Keys>
cudaError_t launch_bounds(const BoundsParams &p, cudaStream_t s)
{
    const size_t smem = (kPrefixScratch + static_cast<size_t>(p.batch) + 1) * sizeof(int32_t);
    const long long warps = static_cast<long long>(p.batch) * p.max_pages * p.hkv;
    long long grid = static_cast<long long>(sm_count()) * 6;
    grid = min(grid, (warps + kBoundThreads / 32 - 1) / (kBoundThreads / 32));
    return launch_pdl(page_bounds_kernel<Keys>, dim3(static_cast<unsigned>(grid)), dim3(kBoundThreads), smem, s, p);
}

// ---- scores --------------------------------------------------------------------

constexpr int kScoreThreads = 256, kScoreWarps = kScoreThreads / 32;
constexpr int kTile = 16;                // pages of one matrix instruction

// D(16x8 s32) += A(16x32 s8, row) * B(32x8 s8, col).
__device__ __forceinline__ void mma_s8_16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pages that query token t of a sequence of length len sees.
__device__ __forceinline__ int pages_seen(int len, int q_len, int t)
{
    const int n = len - q_len + t + 1;
    return n > 0 ? (n + kPageSize - 1) / kPageSize : 0;
}

// The CTAs take equal runs of the (sequence, kv head)s' tiles of 16 pages; a
// CTA's warps take the tiles of its run in turn.  A lane (gid, tig) holds bytes
// 16 tig + 64 i .. + 15, i = 0 .. 3, of the bounds of pages gid and gid + 8: four
// 16-byte loads a page, straight into the operand (its K order is free as long as
// the queries', laid out in shared memory once a (sequence, kv head), is the
// same).  A tile's bounds serve all query tokens.
__global__ void __launch_bounds__(kScoreThreads) page_scores_kernel(const __grid_constant__ SelectParams p)
{
    extern __shared__ __align__(16) uint8_t ssmem[];
    uint4 *frag = reinterpret_cast<uint4 *>(ssmem);              // [q_len][4][32 lanes]
    int32_t *scratch = reinterpret_cast<int32_t *>(frag + p.q_len * 128), *prefix = scratch + kPrefixScratch;
    pdl_wait();
    pdl_launch_dependents();
    const int max_len = p.max_pages * kPageSize;
    build_prefix_of(
        [&](int b) {
            const int len = __ldg(p.seq_lens + b);
            if (blockIdx.x == 0 && (len < 0 || len > max_len))
                report(p.dev_status, NVFP4KV_DEV_BAD_LEN);
            const int pages = (clamp_len(len, max_len) + kPageSize - 1) / kPageSize;
            // (where every page is taken anyway no score is asked for)
            return pages > p.budget ? p.hkv * ((pages + kTile - 1) / kTile) : 0;
        },
        p.batch, prefix, scratch);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const long long total = prefix[p.batch];
    int at = static_cast<int>(total * blockIdx.x / gridDim.x);
    const int end = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
    while (at < end) {
        const int b = find_seq(prefix, p.batch, at);
        const int tiles = (prefix[b + 1] - prefix[b]) / p.hkv;
        const int h = (at - prefix[b]) / tiles, tile0 = at - prefix[b] - h * tiles;
        const int stop = min(tiles, tile0 + end - at);           // of this (sequence, kv head)
        const int len = clamp_len(__ldg(p.seq_lens + b), max_len);
        const int pages = (len + kPageSize - 1) / kPageSize;
        __syncthreads();                                         // the last queries are done with
        // the queries, a warp a token: lane (head gid, channels 16 tig + 64 i ..)
        for (int t = warp; t < p.q_len; t += kScoreWarps) {
            // (columns past the group repeat its last head)
            const uint16_t *q = p.q + ((static_cast<size_t>(b) * p.q_len + t) * p.hq + h * p.group + min(gid, p.group - 1)) *
                                          kHeadDim;
            float x[32], top = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(q + 64 * i + 16 * tig) + k);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        x[16 * i + 8 * k + 2 * m] = __uint_as_float(w[m] << 16);
                        x[16 * i + 8 * k + 2 * m + 1] = __uint_as_float(w[m] & 0xffff0000u);
                    }
                }
#pragma unroll
            for (int k = 0; k < 32; ++k)
                top = fmaxf(top, fabsf(x[k]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
            const float r = top > 0.f ? __fdiv_rn(127.f, top) : 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t pos[4], neg[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    pos[m] = neg[m] = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int w = static_cast<int>(fminf(fmaxf(rintf(__fmul_rn(x[16 * i + 4 * m + k], r)), -127.f), 127.f));
                        pos[m] |= (static_cast<uint32_t>(max(w, 0)) & 0xffu) << (8 * k);
                        neg[m] |= (static_cast<uint32_t>(min(w, 0)) & 0xffu) << (8 * k);
                    }
                }
                // bytes 0 .. 127 of the bounds are the least keys
                frag[(t * 4 + i) * 32 + lane] = make_uint4(neg[0], neg[1], neg[2], neg[3]);
                frag[(t * 4 + 2 + i) * 32 + lane] = make_uint4(pos[0], pos[1], pos[2], pos[3]);
            }
        }
        __syncthreads();
        const int32_t *table = p.block_table + static_cast<size_t>(b) * p.max_pages;
        for (int tile = tile0 + warp; tile < stop; tile += kScoreWarps) {
            const int page = tile * kTile + (lane & 15);
            int phys = page < pages ? __ldg(table + page) : 0;
            if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_pages)) {
                report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);
                phys = 0;
            }
            const size_t head = static_cast<size_t>(phys) * p.hkv + h;
            const float step = __ldg(p.steps + head);
            uint4 a[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int src = __shfl_sync(kFullMask, phys, gid + 8 * r);
                const uint4 *d = reinterpret_cast<const uint4 *>(p.bounds + (static_cast<size_t>(src) * p.hkv + h) *
                                                                                (2 * kHeadDim)) + tig;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a[r][i] = __ldg(d + 4 * i);
            }
            for (int t = 0; t < p.q_len; ++t) {
                int d0[4] = {0, 0, 0, 0}, d1[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 w = frag[(t * 4 + i) * 32 + lane];
                    mma_s8_16832(d0, a[0][i].x, a[1][i].x, a[0][i].y, a[1][i].y, w.x, w.y);
                    mma_s8_16832(d1, a[0][i].z, a[1][i].z, a[0][i].w, a[1][i].w, w.z, w.w);
                }
                int lo = max(d0[0] + d1[0], d0[1] + d1[1]), hi = max(d0[2] + d1[2], d0[3] + d1[3]);
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    lo = max(lo, __shfl_xor_sync(kFullMask, lo, o));
                    hi = max(hi, __shfl_xor_sync(kFullMask, hi, o));
                }
                // row gid's sum is in lanes 4 gid ..; lane l < 16 stores page l's
                const int s0 = __shfl_sync(kFullMask, lo, 4 * (lane & 7)), s1 = __shfl_sync(kFullMask, hi, 4 * (lane & 7));
                if (lane < 16 && page < pages)
                    p.scores[((static_cast<size_t>(b) * p.q_len + t) * p.hkv + h) * p.score_stride + page] =
                        __fmul_rn(static_cast<float>(lane < 8 ? s0 : s1), step);
            }
        }
        at += stop - tile0;
    }
}

// ---- selection -----------------------------------------------------------------

constexpr int kPickThreads = 512, kPickWarps = kPickThreads / 32;
constexpr int kBins = 2048;
constexpr int kTies = 1024;              // scores of the border's bin that are ranked side by side

// A float's place in the order of floats, as an unsigned number.
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float float_at(uint32_t place)
{
    return __uint_as_float(place & 0x80000000u ? place & 0x7fffffffu : ~place);
}

// Exclusive sum over the CTA of one value a thread; the total in `total`.
__device__ __forceinline__ int cta_sum_before(int v, int32_t *scratch, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFullMask, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        scratch[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int i = 0; i < kPickWarps; ++i) {
        before += i < warp ? scratch[i] : 0;
        total += scratch[i];
    }
    return before + x - v;
}

// One CTA a (query token, kv head).  Counts of the scores in 2,048 equal parts of
// [least, largest] say, from the top, in which part the last wanted one lies; what
// lies above is taken, what lies in that part is ranked pair by pair.  (The part
// of a score never falls as the score grows, whatever its subtraction and product
// round.)  Where more than kTies scores share the part, it is cut into 2,048
// again, by the order of floats, until they fit or are one number, of which the
// lowest pages are taken.
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const __grid_constant__ SelectParams p)
{
    extern __shared__ uint32_t taken[];                          // a bit a page
    __shared__ int32_t scratch[kPickWarps], count[kBins];
    __shared__ uint32_t tie_key[kTies];
    __shared__ int32_t tie_page[kTies];
    __shared__ uint32_t edge[2];
    __shared__ int32_t found[3];
    const int tid = threadIdx.x, lane = tid & 31;
    const long long unit = blockIdx.x;                           // (sequence, token, kv head)
    const long long row = unit / p.hkv;
    const int b = static_cast<int>(row / p.q_len), t = static_cast<int>(row - static_cast<long long>(b) * p.q_len);
    pdl_wait();
    pdl_launch_dependents();
    const int pages = pages_seen(clamp_len(__ldg(p.seq_lens + b), p.max_pages * kPageSize), p.q_len, t);
    int32_t *out = p.pages + unit * p.budget;
    if (pages <= p.budget) {
        for (int i = tid; i < p.budget; i += kPickThreads)
            out[i] = i < pages ? i : -1;
        return;
    }
    const float *score = p.scores + unit * p.score_stride;
    const int lo = p.first, hi = pages - p.last;                 // the candidates
    int want = p.budget - p.first - p.last;                      // fewer than there are
    const int words = (pages + 31) / 32;
    for (int i = tid; i < words; i += kPickThreads)
        taken[i] = 0;
    // fn(page, its score's place in the order of floats)
    auto for_scores = [&](auto fn) {
        for (int i = lo + tid; i < hi; i += kPickThreads)
            fn(i, order_of(__ldcg(score + i)));
    };
    // edge: the least and the largest of those that in(place) holds for
    auto find_edges = [&](auto in) {
        uint32_t least = 0xffffffffu, most = 0;
        __syncthreads();
        if (tid == 0) {
            edge[0] = 0xffffffffu;
            edge[1] = 0;
        }
        __syncthreads();
        for_scores([&](int, uint32_t k) {
            if (in(k)) {
                least = min(least, k);
                most = max(most, k);
            }
        });
        least = __reduce_min_sync(kFullMask, least);
        most = __reduce_max_sync(kFullMask, most);
        if (lane == 0) {
            atomicMin(edge, least);
            atomicMax(edge + 1, most);
        }
        __syncthreads();
    };
    find_edges([](uint32_t) { return true; });
    uint32_t from = edge[0], to = edge[1];                       // the places that are still open, both ends among them
    bool equal_parts = true;                                     // of numbers; later, of places
    while (want > 0 && from < to) {
        const float base = float_at(from), by = kBins / (float_at(to) - base);
        const uint32_t span = to - from;
        const int shift = span < kBins ? 0 : 21 - __clz(span);   // at most 2,048 parts of 2^shift places
        auto part_of = [&](uint32_t k) {                         // -1 under the open ones, kBins above
            if (k < from || k > to)
                return k < from ? -1 : kBins;
            return equal_parts ? static_cast<int>(fminf(fmaxf((float_at(k) - base) * by, 0.f), kBins - 1.f))
                               : static_cast<int>((k - from) >> shift);
        };
        __syncthreads();
        for (int i = tid; i < kBins; i += kPickThreads)
            count[i] = 0;
        if (tid == 0)
            found[2] = 0;
        __syncthreads();
        for_scores([&](int, uint32_t k) {
            const int part = part_of(k);
            if (part >= 0 && part < kBins)
                atomicAdd(&count[part], 1);
        });
        __syncthreads();
        // the part where the count from the top reaches `want`
        int mine[kBins / kPickThreads], sum = 0, total;
        const int top = kBins - 1 - tid * (kBins / kPickThreads);
#pragma unroll
        for (int k = 0; k < kBins / kPickThreads; ++k) {
            mine[k] = count[top - k];
            sum += mine[k];
        }
        int before = cta_sum_before(sum, scratch, total);
#pragma unroll
        for (int k = 0; k < kBins / kPickThreads; ++k) {
            if (before < want && want <= before + mine[k]) {
                found[0] = top - k;
                found[1] = before;
            }
            before += mine[k];
        }
        __syncthreads();
        const int border = found[0], inside = count[border];
        want -= found[1];
        const bool whole = inside == want, rank = !whole && inside <= kTies;
        for_scores([&](int i, uint32_t k) {
            const int part = part_of(k);
            if (part < border || part == kBins)                  // (above the open ones: taken in an earlier turn)
                return;
            if (part > border || whole) {
                atomicOr(&taken[i >> 5], 1u << (i & 31));
            } else if (rank) {
                const int n = atomicAdd(&found[2], 1);
                tie_key[n] = k;
                tie_page[n] = i;
            }
        });
        __syncthreads();
        if (rank)
            for (int x = tid; x < inside; x += kPickThreads) {
                const uint32_t k = tie_key[x];
                const int page = tie_page[x];
                int r = 0;
                for (int y = 0; y < inside; ++y)
                    r += tie_key[y] > k || (tie_key[y] == k && tie_page[y] < page);
                if (r < want)
                    atomicOr(&taken[page >> 5], 1u << (page & 31));
            }
        if (whole || rank) {
            want = 0;
        } else {
            find_edges([&](uint32_t k) { return part_of(k) == border; });
            from = edge[0];
            to = edge[1];
            equal_parts = false;
        }
    }
    // (one number left) the lowest `want` of the pages that have it
    for (int i0 = lo; i0 < hi && want > 0; i0 += kPickThreads) {
        const int i = i0 + tid;
        const bool is = i < hi && order_of(__ldcg(score + i)) == from;
        int total;
        const int before = cta_sum_before(is, scratch, total);
        if (is && before < want)
            atomicOr(&taken[i >> 5], 1u << (i & 31));
        want -= total;
    }
    __syncthreads();
    // the list, ascending
    int done = 0;
    for (int w0 = 0; w0 < words; w0 += kPickThreads) {
        const int w = w0 + tid;
        uint32_t bits = 0;
        if (w < words) {
            bits = taken[w];
            const int p0 = 32 * w;
            // first pages, and last ones
            bits |= p0 + 32 <= p.first ? 0xffffffffu : (p0 < p.first ? (1u << (p.first - p0)) - 1u : 0u);
            const uint32_t below = hi >= p0 + 32 ? 0xffffffffu : (hi > p0 ? (1u << (hi - p0)) - 1u : 0u);
            const uint32_t there = pages >= p0 + 32 ? 0xffffffffu : (1u << (pages - p0)) - 1u;
            bits |= there & ~below;
        }
        int total;
        int n = done + cta_sum_before(__popc(bits), scratch, total);
        while (bits) {
            const int k = __ffs(bits) - 1;
            bits &= bits - 1;
            out[n++] = 32 * w + k;
        }
        done += total;
    }
}

} // namespace

cudaError_t launch_page_bounds_nvfp4(const BoundsParams &p, cudaStream_t s)
{
    return launch_bounds<Nvfp4Keys>(p, s);
}

cudaError_t launch_page_bounds_fp8_block(const BoundsParams &p, cudaStream_t s)
{
    return launch_bounds<Fp8BlockKeys>(p, s);
}

int score_row_stride(int max_pages)
{
    return (max_pages + kTile - 1) / kTile * kTile;
}

cudaError_t launch_select_pages(const SelectParams &p, cudaStream_t s)
{
    const size_t smem = static_cast<size_t>(p.q_len) * 4 * 32 * sizeof(uint4) +
                        (kPrefixScratch + static_cast<size_t>(p.batch) + 1) * sizeof(int32_t);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(page_scores_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess)
            return e;
    }
    const long long tiles = static_cast<long long>(p.batch) * p.hkv * ((p.max_pages + kTile - 1) / kTile);
    long long grid = static_cast<long long>(sm_count()) * 3;
    grid = max(1LL, min(grid, (tiles + kScoreWarps - 1) / kScoreWarps));
    cudaError_t e = launch_pdl(page_scores_kernel, dim3(static_cast<unsigned>(grid)), dim3(kScoreThreads), smem, s, p);
    if (e != cudaSuccess)
        return e;
    const size_t bits = (static_cast<size_t>(p.max_pages) + 31) / 32 * 4;
    if (bits > 16 * 1024) {
        e = cudaFuncSetAttribute(page_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bits));
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(page_pick_kernel, dim3(static_cast<unsigned>(p.batch * p.q_len * p.hkv)), dim3(kPickThreads), bits, s,
                      p);
}

} // namespace nvfp4kv
