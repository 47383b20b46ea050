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
// (w+, w-) . (hi, lo), which runs on the tensor cores.
// A query takes the first pages and the last ones of its sequence and, of the
// others, those of the largest scores, the lower page first where they tie.
#include "cluster.cuh"
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

// Keys of a page-head by lane: lane l holds channels 8c .. 8c + 7, c = l mod 16,
// of the tokens 2i + floor(l / 16), i = 0 .. 7.  A value is x[i] * unit().
struct Nvfp4Keys {
    static constexpr int kRecord = kNvfp4Record;
    uint32_t d[8], s[8];

    __device__ __forceinline__ void load(const uint8_t *rec, int lane)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            d[i] = reinterpret_cast<const uint32_t *>(rec)[32 * i + lane];
            s[i] = rec[2048 + 16 * i + 8 * (lane >> 4) + ((lane & 15) >> 1)];
        }
    }
    // The scale byte's seven bits moved to f16's exponent and mantissa are the
    // scale times 2^-8 without a conversion; times a code's value it is exact.
    __device__ __forceinline__ float unit() const { return 256.f; }
    __device__ __forceinline__ void get(int i, uint32_t (&x)[4]) const
    {
        const uint32_t sc = s[i] * 0x00800080u;
        e2m1x8_to_f16x2x4(d[i], x[0], x[1], x[2], x[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k] = hmul2(x[k], sc);
    }
};

struct Fp8BlockKeys {
    static constexpr int kRecord = kFp8BlockRecord;
    uint2 d[8];
    float s;

    __device__ __forceinline__ void load(const uint8_t *rec, int lane)
    {
        // (the chunk of 16 channels is one place further in odd rows)
        const int place = 2 * ((((lane & 15) >> 1) + (lane >> 4)) & 7) + (lane & 1);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            d[i] = reinterpret_cast<const uint2 *>(rec)[32 * i + (lane & 16) + place];
        s = *reinterpret_cast<const float *>(rec + kFp8Record);
    }
    __device__ __forceinline__ float unit() const { return s; }
    __device__ __forceinline__ void get(int i, uint32_t (&x)[4]) const
    {
        e4m3x4_to_f16x2x2(d[i].x, x[0], x[1]);
        e4m3x4_to_f16x2x2(d[i].y, x[2], x[3]);
    }
};

// 1.5 * 2^23: a sum with it, rounded up or down, has the whole number in its low
// byte, as two's complement.
constexpr float kWhole = 12582912.f;

// The bounds of one page-head by a warp.  All arithmetic in fp32 is on x, the
// values over unit(), a power of two: fl32(x * fl32(127 / max |x|)) is what the
// definition has for k = x * unit.
template <class Keys>
__device__ __forceinline__ void write_bounds(const Keys &keys, int valid, int8_t *dst, float *step, int lane)
{
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        lo[k] = 0x7c007c00u;                                     // +inf, -inf
        hi[k] = 0xfc00fc00u;
    }
    auto take = [&](int i) {
        uint32_t x[4];
        keys.get(i, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            lo[k] = hmin2(lo[k], x[k]);
            hi[k] = hmax2(hi[k], x[k]);
        }
    };
    if (valid >= kPageSize) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            take(i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (2 * i + (lane >> 4) < valid)
                take(i);
    }
    // even and odd tokens meet; each lane keeps four of its eight channels
    const bool upper = lane & 16;
    uint32_t l[2], h[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t lo_away = upper ? lo[k] : lo[k + 2], hi_away = upper ? hi[k] : hi[k + 2];
        l[k] = hmin2(upper ? lo[k + 2] : lo[k], __shfl_xor_sync(kFullMask, lo_away, 16));
        h[k] = hmax2(upper ? hi[k + 2] : hi[k], __shfl_xor_sync(kFullMask, hi_away, 16));
    }
    uint32_t t2 = hmax2(hmax2(l[0] & 0x7fff7fffu, l[1] & 0x7fff7fffu), hmax2(h[0] & 0x7fff7fffu, h[1] & 0x7fff7fffu));
    // (f16 numbers that are not negative are in the order of their bits)
    t2 = __reduce_max_sync(kFullMask, max(t2 & 0xffffu, t2 >> 16));
    const float top = __half2float(__ushort_as_half(static_cast<unsigned short>(t2)));
    // one division: 127 / top in the lower half warp, top / 127 in the upper one
    const float quot = __fdiv_rn(upper ? top : 127.f, upper ? 127.f : top);
    const float r = top > 0.f ? __shfl_sync(kFullMask, quot, 0) : 0.f;
    uint32_t wl[4], wh[4];
    const uint64_t r2 = f32x2_pack(r, r), whole2 = f32x2_pack(kWhole, kWhole);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&l[k]));
        const float2 d = __half22float2(*reinterpret_cast<__half2 *>(&h[k]));
        uint64_t lo2, hi2;
        asm("add.rm.f32x2 %0, %1, %2;" : "=l"(lo2) : "l"(mul_f32x2(f32x2_pack(a.x, a.y), r2)), "l"(whole2));
        asm("add.rp.f32x2 %0, %1, %2;" : "=l"(hi2) : "l"(mul_f32x2(f32x2_pack(d.x, d.y), r2)), "l"(whole2));
        wl[2 * k] = __float_as_uint(fmaxf(f32x2_lo(lo2), kWhole - 127.f));
        wl[2 * k + 1] = __float_as_uint(fmaxf(f32x2_hi(lo2), kWhole - 127.f));
        wh[2 * k] = __float_as_uint(fminf(f32x2_lo(hi2), kWhole + 127.f));
        wh[2 * k + 1] = __float_as_uint(fminf(f32x2_hi(hi2), kWhole + 127.f));
    }
    auto bytes = [](const uint32_t (&w)[4]) {
        return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
    };
    int8_t *at = dst + 8 * (lane & 15) + (upper ? 4 : 0);
    *reinterpret_cast<uint32_t *>(at) = bytes(wl);
    *reinterpret_cast<uint32_t *>(at + kHeadDim) = bytes(wh);
    if (lane == 16)
        *step = quot * keys.unit();
}

// One warp a page, or a part of its heads where there are fewer pages than warps.
// Bound by its instructions more than by memory, half of them the expansion to f16 and
// the two comparisons a pair of values: 15 prompts of 32K at 8 heads take 77 us for 304
// MB.  So many warps rather than loads ahead of their use: with the next head's keys in
// registers, 32 warps an SM instead of 48, 81 us.  More CTAs than run at a time, for the
// last pages' sake (8 an SM, 6 of which run; with 4, which are not placed evenly, 117).
template <class Keys>
__global__ void __launch_bounds__(kBoundThreads, 6) page_bounds_kernel(const __grid_constant__ BoundsParams p)
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
    const int pages = prefix[p.batch], warps = gridDim.x * (kBoundThreads / 32);
    if (pages == 0)
        return;
    const int parts = min(p.hkv, max(1, warps / pages));
    const long long units = static_cast<long long>(pages) * parts;
    for (long long u = blockIdx.x * (kBoundThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const int pg = parts == 1 ? static_cast<int>(u) : static_cast<int>(u / parts);
        const int part = static_cast<int>(u - static_cast<long long>(pg) * parts);
        const int b = find_seq(prefix, p.batch, pg);
        const int len = clamp_len(__ldg(p.seq_lens + b), max_len);
        const int page = first_page(b, len) + pg - prefix[b];
        const int phys = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + page);
        if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_pages)) {
            if (part == 0 && lane == 0)
                report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);
            continue;
        }
        const int valid = len - page * kPageSize;
        const int h0 = static_cast<int>(static_cast<long long>(p.hkv) * part / parts);
        const int h1 = static_cast<int>(static_cast<long long>(p.hkv) * (part + 1) / parts);
        size_t head = static_cast<size_t>(phys) * p.hkv + h0;
        const uint8_t *rec = p.pool + head * Keys::kRecord;
        for (int h = h0; h < h1; ++h, ++head, rec += Keys::kRecord) {
            Keys keys;
            keys.load(rec, lane);
            write_bounds(keys, valid, p.bounds + head * (2 * kHeadDim), p.steps + head, lane);
        }
    }
}

template <class Keys>
cudaError_t launch_bounds(const BoundsParams &p, cudaStream_t s)
{
    const size_t smem = (kPrefixScratch + static_cast<size_t>(p.batch) + 1) * sizeof(int32_t);
    const long long warps = static_cast<long long>(p.batch) * p.max_pages * p.hkv;
    long long grid = static_cast<long long>(sm_count()) * 8;
    grid = min(grid, (warps + kBoundThreads / 32 - 1) / (kBoundThreads / 32));
    return launch_pdl(page_bounds_kernel<Keys>, dim3(static_cast<unsigned>(grid)), dim3(kBoundThreads), smem, s, p);
}

// ---- scores --------------------------------------------------------------------

constexpr int kTile = 16;                // pages of one matrix instruction

// Queries of a token and kv head as operands: a token's are kQueryWords uint4 --
// [8][32 lanes] of f16 pairs, then what each of the eight heads' sums starts from.
constexpr int kQueryWords = 8 * 32 + 2;

// Pages that query token t of a sequence of length len sees.
__device__ __forceinline__ int pages_seen(int len, int q_len, int t)
{
    const int n = len - q_len + t + 1;
    return n > 0 ? (n + kPageSize - 1) / kPageSize : 0;
}

// The queries of a token and kv head in whole steps, by a warp: lane (head gid,
// channels 16 tig + 64 i .. + 15, i = 0, 1).
__device__ __forceinline__ void load_queries(const SelectParams &p, int b, int t, int h, uint4 *frag, int lane)
{
    const int gid = lane >> 2, tig = lane & 3;
    // (columns past the group repeat its last head)
    const uint16_t *q = p.q + ((static_cast<size_t>(b) * p.q_len + t) * p.hq + h * p.group + min(gid, p.group - 1)) *
                                  kHeadDim;
    float x[32], top = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint4 v = reinterpret_cast<const uint4 *>(q + 64 * i + 16 * tig)[k];
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
    if (top < 0x1p-100f) {
        // (127 / top might pass fp32: the same weights of queries 2^100 times as large)
        top *= 0x1p100f;
#pragma unroll
        for (int k = 0; k < 32; ++k)
            x[k] *= 0x1p100f;
    }
    const float r = top > 0.f ? __fdiv_rn(127.f, top) : 0.f;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint32_t pos[4], neg[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float w[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    w[e] = fminf(fmaxf(rintf(__fmul_rn(x[16 * i + 8 * m + 2 * k + e], r)), -127.f), 127.f);
                    sum += static_cast<int>(w[e]);
                }
                pos[k] = pack_f16x2(fmaxf(w[0], 0.f), fmaxf(w[1], 0.f));
                neg[k] = pack_f16x2(fminf(w[0], 0.f), fminf(w[1], 0.f));
            }
            // bytes 0 .. 127 of the bounds are the least keys
            frag[(2 * i + m) * 32 + lane] = make_uint4(neg[0], neg[1], neg[2], neg[3]);
            frag[(4 + 2 * i + m) * 32 + lane] = make_uint4(pos[0], pos[1], pos[2], pos[3]);
        }
    sum += __shfl_xor_sync(kFullMask, sum, 1);
    sum += __shfl_xor_sync(kFullMask, sum, 2);
    if (tig == 0)
        reinterpret_cast<float *>(frag + 8 * 32)[gid] = static_cast<float>(-128 * sum) * 0x1p-24f;
}

// A warp's ring of tiles in shared memory, copied 16 bytes a lane, so that what is in
// flight takes no registers.  (Bulk copies of a page's 256 bytes each came in at 43
// GB/s an SM: one in 11 cycles.)  Pages 2r and 2r + 1 of a tile lie 320 bytes apart
// and the next pair 576 further, so that the eight lanes of a read, four a page, meet
// different banks.
constexpr int kStages = 2;
constexpr uint32_t kStageBytes = 8 * 576;

struct TileRing {
    uint32_t data;                       // shared-memory address
    float step[kStages];                 // of page lane mod 16 of each stage's tile

    // Asks for the tile whose page ids lanes l and l + 16 hold for page l; with
    // `there` false for nothing.  One call a turn, so that the turns can be counted.
    __device__ __forceinline__ void ask(const SelectParams &p, int h, bool there, int phys, int stage, int lane)
    {
        if (there) {
            __syncwarp();                // (the stage has been read)
            const uint32_t dst = data + stage * kStageBytes + (lane >> 4) * 320 + (lane & 15) * 16;
#pragma unroll
            for (int k = 0; k < kTile / 2; ++k) {
                const int id = __shfl_sync(kFullMask, phys, 2 * k + (lane >> 4));
                const int8_t *src = p.bounds + (static_cast<size_t>(id) * p.hkv + h) * (2 * kHeadDim) + (lane & 15) * 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + k * 576), "l"(src) : "memory");
            }
            step[stage] = p.steps[static_cast<size_t>(phys) * p.hkv + h];
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    // Waits for the oldest tile asked for.
    __device__ __forceinline__ void wait() const
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
    }

    // The stage's tile into registers, after which the stage is free: a lane (gid,
    // tig) takes bytes 16 tig + 64 i .. + 15, i = 0 .. 3, of pages gid and gid + 8
    // (the operand's K order is free as long as the queries' is the same).
    __device__ __forceinline__ void read(int stage, uint4 (&a)[2][4], int lane) const
    {
        const int gid = lane >> 2;
        const uint32_t at = data + stage * kStageBytes + (gid >> 1) * 576 + (gid & 1) * 320 + 16 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[0][i] = lds128(at + 64 * i);
            a[1][i] = lds128(at + 4 * 576 + 64 * i);
        }
    }
};

// The score of a tile's page lane mod 16; query(i): the queries' word i of the lane,
// from: what the sums of heads 2tig and 2tig + 1 start from.  (8-bit integer matrix
// instructions: three tokens and more a sequence take 1.4 times as long.)  A byte plus
// 128, with a zero byte above it, is the f16 number (byte + 128) * 2^-24: two
// permutations for four bytes.  The sums start from -128 sum w and are exact multiples
// of 2^-24 below 1.  What no bounds of finite keys give (a step that is NaN or
// infinite) is held to finite numbers.
template <class Query>
__device__ __forceinline__ float score_of(const uint4 (&tile)[2][4], Query query, float2 from, float step, int lane)
{
    float d[4][4] = {{from.x, from.y, from.x, from.y}, {0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 w0 = query(2 * i), w1 = query(2 * i + 1);
        const uint32_t a[4] = {tile[0][i].x, tile[0][i].y, tile[0][i].z, tile[0][i].w};
        const uint32_t b[4] = {tile[1][i].x, tile[1][i].y, tile[1][i].z, tile[1][i].w};
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t x = a[k] ^ 0x80808080u, y = b[k] ^ 0x80808080u;
            mma_f16_16816(d[k], __byte_perm(x, 0, 0x4140), __byte_perm(y, 0, 0x4140), __byte_perm(x, 0, 0x4342),
                          __byte_perm(y, 0, 0x4342), w[2 * k], w[2 * k + 1]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        d[0][e] = (d[0][e] + d[1][e]) + (d[2][e] + d[3][e]);
    float lo = fmaxf(d[0][0], d[0][1]), hi = fmaxf(d[0][2], d[0][3]);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lo = fmaxf(lo, __shfl_xor_sync(kFullMask, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(kFullMask, hi, o));
    }
    // page gid's is in lanes 4 gid ..
    const float s0 = __shfl_sync(kFullMask, lo, 4 * (lane & 7)), s1 = __shfl_sync(kFullMask, hi, 4 * (lane & 7));
    constexpr float kLargest = 3.40282347e+38f;
    return fminf(fmaxf(__fmul_rn(((lane & 8) ? s1 : s0) * 0x1p24f, step), -kLargest), kLargest) + 0.f;   // (-0 is 0)
}

// A page id of a table, 0 for one that is not there.
__device__ __forceinline__ int checked(const SelectParams &p, int phys)
{
    if (static_cast<unsigned>(phys) < static_cast<unsigned>(p.num_pages))
        return phys;
    report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);
    return 0;
}

// ---- selection -----------------------------------------------------------------

constexpr int kBins = 2048;
constexpr int kTies = 1024;              // scores of the border's bin that are ranked side by side
static_assert(2 * kTies <= kBins, "all CTAs' ties in the place of a CTA's counts");

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
template <int kThreads>
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
    for (int i = 0; i < kThreads / 32; ++i) {
        before += i < warp ? scratch[i] : 0;
        total += scratch[i];
    }
    return before + x - v;
}

// What the CTAs of a cluster show one another while they select, and a CTA's scratch.
struct alignas(16) PickShared {
    int32_t scratch[32], count[kBins];
    uint32_t tie_key[kTies];
    int32_t tie_page[kTies];
    int32_t found[4];                    // the border's part, scores above it, scores in it; ties that are kept
    uint32_t least, most;                // of this CTA's scores, as places in the order of floats
    uint32_t part_least, part_most;      // ... of those in the border's part
    int32_t equal, listed;               // scores that are the one number left; entries of the list
};

// Ready for the first counts (the CTA meets before they begin).
template <int kThreads>
__device__ __forceinline__ void clear_counts(PickShared &sh)
{
    for (int i = threadIdx.x; i < kBins; i += kThreads)
        sh.count[i] = 0;
    if (threadIdx.x == 0) {
        sh.found[3] = 0;
        sh.part_least = 0xffffffffu;
        sh.part_most = 0;
    }
}

// A query token and kv head's selection, by a cluster: this CTA has the scores of
// pages p0 .. p0 + count - 1 in `score`.
struct Selection {
    const float *score;
    uint32_t *taken;                     // a bit a page of this CTA, all clear
    int p0, count;
    int lo, hi;                          // the candidates among them, as score[lo .. hi - 1]
    int pages, first, last;              // of the sequence; pages that are taken in any case
    uint32_t rank, ranks;
};

// The CTAs of the cluster meet.
__device__ __forceinline__ void meet(uint32_t ranks)
{
    if (ranks > 1)
        cluster_sync();
    else
        __syncthreads();
}

// Finds the `want` best of the candidates, all pages but the first and last ones (there
// are more of them), and lists them with those, ascending, at `out`.  Counts of the
// scores in 2,048 equal parts of [least, largest] say, from the top, in which part the
// last wanted one lies; what lies above is taken, what lies in that part is ranked pair
// by pair.  `from` and `to` are the ends of the thread's scores in the order of floats,
// then of what is still open.  (The part of a score, f below cut to a whole number, never falls as the
// score grows, whatever its difference and product round.)  Where more than kTies
// scores share the part, its places in the order of floats are cut into 2,048 parts,
// again until they fit or are one number, of which the lowest pages are taken.  Every
// CTA adds up all CTAs' counts and comes to the same border.
template <int kThreads>
__device__ __forceinline__ void pick_pages(const Selection &s, uint32_t from, uint32_t to, int want, int32_t *out, PickShared &sh)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t base = smem_addr(&sh);
    auto peer = [&](const void *field, uint32_t k) { return in_cta(base + static_cast<uint32_t>(
        static_cast<const uint8_t *>(field) - reinterpret_cast<const uint8_t *>(&sh)), k); };
    auto for_scores = [&](auto fn) {
#pragma unroll 4
        for (int i = s.lo + tid; i < s.hi; i += kThreads)
            fn(i, s.score[i]);
    };
    // What lane k reads of CTA k, `none` in the lanes past the last one: one trip to
    // the other CTAs for all of them.
    auto of_each = [&](const void *field, uint32_t none) {
        return static_cast<uint32_t>(lane) < s.ranks ? ld_cluster_u32(peer(field, lane)) : none;
    };
    // A place range of the cluster, from each CTA's.
    auto range_of = [&](const uint32_t &least, const uint32_t &most, uint32_t &a, uint32_t &z) {
        if (s.ranks == 1) {
            a = least;
            z = most;
            return;
        }
        const uint32_t x = of_each(&least, 0xffffffffu), y = of_each(&most, 0);
        a = __reduce_min_sync(kFullMask, x);
        z = __reduce_max_sync(kFullMask, y);
    };
    // The sum of what the CTAs before this one have.
    auto before_me = [&](const int32_t &field) {
        if (s.ranks == 1)
            return 0;
        const uint32_t x = of_each(&field, 0);
        return static_cast<int>(__reduce_add_sync(kFullMask, static_cast<uint32_t>(lane) < s.rank ? x : 0u));
    };
    // The part where the count from the top reaches `want`, which loses what lies
    // above; scores in the part.
    int border = 0, inside = 0;
    auto find_border = [&]() {
        meet(s.ranks);
        constexpr int kEach = kBins / kThreads;
        int mine[kEach], sum = 0, total;
        const int top = kBins - 1 - tid * kEach;
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            mine[k] = s.ranks > 1 ? 0 : sh.count[top - k];
        for (uint32_t r0 = 0; s.ranks > 1 && r0 < s.ranks; r0 += 4) {
            uint32_t n[4][kEach];                                // (asked for together)
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r) {
                const uint32_t at = peer(&sh.count[top], min(r0 + r, s.ranks - 1));
#pragma unroll
                for (int k = 0; k < kEach; ++k)
                    n[r][k] = r0 + r < s.ranks ? ld_cluster_u32(at - 4 * k) : 0u;
            }
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r)
#pragma unroll
                for (int k = 0; k < kEach; ++k)
                    mine[k] += static_cast<int>(n[r][k]);
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            sum += mine[k];
        int before = cta_sum_before<kThreads>(sum, sh.scratch, total);
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (before < want && want <= before + mine[k]) {
                sh.found[0] = top - k;
                sh.found[1] = before;
                sh.found[2] = mine[k];
            }
            before += mine[k];
        }
        __syncthreads();
        border = sh.found[0];
        inside = sh.found[2];
        want -= sh.found[1];
    };
    auto take = [&](int i) { atomicOr(&s.taken[i >> 5], 1u << (i & 31)); };
    // A score in the border's part: taken with all of it, kept to be ranked, or only
    // noted in the part's range.
    auto at_border = [&](int i, float x) {
        const uint32_t k = order_of(x);
        if (inside == want) {
            take(i);
        } else if (inside <= kTies) {
            const int n = atomicAdd(&sh.found[3], 1);
            sh.tie_key[n] = k;
            sh.tie_page[n] = s.p0 + i;
        } else {
            atomicMin(&sh.part_least, k);
            atomicMax(&sh.part_most, k);
        }
    };
    // What is left of the border's part; false when it is still to be cut.
    auto finish = [&]() {
        meet(s.ranks);
        if (inside == want)
            return true;
        if (inside > kTies)
            return false;
        const uint32_t *keys = sh.tie_key;
        const int32_t *at = sh.tie_page;
        if (s.ranks > 1) {
            // all CTAs' ties, in the place of the counts, which have been read
            uint32_t *to = reinterpret_cast<uint32_t *>(sh.count);
            uint32_t end = of_each(&sh.found[3], 0);             // where CTA `lane`'s end among them all
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                const uint32_t x = __shfl_up_sync(kFullMask, end, o);
                end += lane >= o ? x : 0u;
            }
            for (int x0 = 0; x0 < inside; x0 += kThreads) {
                const int x = x0 + tid;
                uint32_t c = 0, begin = 0;
#pragma unroll
                for (int k = 0; k < 7; ++k) {
                    const uint32_t e = __shfl_sync(kFullMask, end, k);
                    if (static_cast<uint32_t>(x) >= e) {
                        c = k + 1;
                        begin = e;
                    }
                }
                if (x < inside && c < s.ranks) {
                    to[x] = ld_cluster_u32(peer(sh.tie_key, c) + 4 * (x - begin));
                    to[kTies + x] = ld_cluster_u32(peer(sh.tie_page, c) + 4 * (x - begin));
                }
            }
            keys = to;
            at = reinterpret_cast<const int32_t *>(to + kTies);
            __syncthreads();
        }
        for (int x = tid; x < inside; x += kThreads) {
            const uint32_t k = keys[x];
            const int page = at[x], i = page - s.p0;
            if (i < 0 || i >= s.count)
                continue;                                        // (another CTA's)
            int r = 0;
#pragma unroll 4
            for (int y = 0; y < inside; ++y)
                r += keys[y] > k || (keys[y] == k && at[y] < page);
            if (r < want)
                take(i);
        }
        return true;
    };

    from = __reduce_min_sync(kFullMask, from);
    to = __reduce_max_sync(kFullMask, to);
    if (lane == 0) {
        atomicMin(&sh.least, from);
        atomicMax(&sh.most, to);
    }
    meet(s.ranks);
    range_of(sh.least, sh.most, from, to);
    bool done = want <= 0;
    if (!done && from < to) {
        // Halves, whose difference is finite whatever the scores, in the same arithmetic for
        // both passes: a score that is counted in one part and found in another would be
        // missed, or be one more than the ties that there is room for.  (Scores so close
        // that `by` is infinite all come to the last part: 0 times it is NaN, which the
        // clamp turns into it and no comparison with a border holds for.)
        const float half = 0.5f * float_at(from), by = kBins / __fmaf_rn(0.5f, float_at(to), -half);
        auto place_of = [&](float x) { return __fmul_rn(__fmaf_rn(0.5f, x, -half), by); };
        for_scores([&](int, float x) {
            const int part = static_cast<int>(fminf(place_of(x), kBins - 1.f));
            atomicAdd(&sh.count[part & (kBins - 1)], 1);
        });
        find_border();
        const float below = border > 0 ? static_cast<float>(border) : -INFINITY;
        const float above = border < kBins - 1 ? static_cast<float>(border + 1) : NAN;
        for_scores([&](int i, float x) {
            const float f = place_of(x);
            if (f >= above)
                take(i);
            else if (!(f < below))
                at_border(i, x);
        });
        done = finish();
        if (!done)
            range_of(sh.part_least, sh.part_most, from, to);
    }
    while (!done && from < to) {
        const uint32_t span = to - from;
        const int shift = span < kBins ? 0 : 21 - __clz(span);   // at most 2,048 parts of 2^shift places
        meet(s.ranks);                                           // (the counts and the range have been read)
        clear_counts<kThreads>(sh);
        __syncthreads();
        for_scores([&](int, float x) {
            const uint32_t k = order_of(x);
            if (k >= from && k <= to)
                atomicAdd(&sh.count[(k - from) >> shift], 1);
        });
        find_border();
        const uint32_t b0 = from + (static_cast<uint32_t>(border) << shift);
        const uint32_t b1 = min(to, b0 + ((1u << shift) - 1u));
        for_scores([&](int i, float x) {
            const uint32_t k = order_of(x);
            if (k > b1 && k <= to)                               // (above the open ones: taken in an earlier turn)
                take(i);
            else if (k >= b0 && k <= b1)
                at_border(i, x);
        });
        done = finish();
        from = b0;
        to = b1;
    }
    if (!done) {
        // one number left: the lowest `want` of the pages that have it
        int n = 0, total;
        for (int i = s.lo + tid; i < s.hi; i += kThreads)
            n += order_of(s.score[i]) == from;
        __syncthreads();
        cta_sum_before<kThreads>(n, sh.scratch, total);
        if (tid == 0)
            sh.equal = total;
        meet(s.ranks);
        want -= before_me(sh.equal);
        for (int i0 = s.lo; i0 < s.hi && want > 0; i0 += kThreads) {
            const int i = i0 + tid;
            const bool is = i < s.hi && order_of(s.score[i]) == from;
            const int before = cta_sum_before<kThreads>(is, sh.scratch, total);
            if (is && before < want)
                take(i);
            want -= total;
        }
    }
    __syncthreads();
    // the list, ascending: first how many entries each CTA has
    auto word = [&](int w) {
        uint32_t bits = s.taken[w];
        const int page = s.p0 + 32 * w, held = s.count - 32 * w;
        auto under = [](int n) { return n >= 32 ? 0xffffffffu : (n > 0 ? (1u << n) - 1u : 0u); };
        bits |= under(s.first - page) | ~under(s.pages - s.last - page);
        return bits & under(held);
    };
    const int words = (s.count + 31) / 32;
    int n0 = 0, total;
    if (s.ranks > 1) {
        for (int w = tid; w < words; w += kThreads)
            n0 += __popc(word(w));
        cta_sum_before<kThreads>(n0, sh.scratch, total);
        if (tid == 0)
            sh.listed = total;
        meet(s.ranks);
        n0 = before_me(sh.listed);
    }
    constexpr int kWarps = kThreads / 32;
    for (int w0 = 0; w0 < words;) {
        const int each = min((words - w0 + kWarps - 1) / kWarps, 32);        // words of a warp
        const int w = w0 + (tid >> 5) * each + lane;
        const uint32_t bits = lane < each && w < words ? word(w) : 0;
        const int n = n0 + cta_sum_before<kThreads>(__popc(bits), sh.scratch, total);
        for (int k = 0; k < each; ++k) {                         // a lane a page
            const uint32_t x = __shfl_sync(kFullMask, bits, k);
            const int at = __shfl_sync(kFullMask, n, k);
            if (x >> lane & 1)
                out[at + __popc(x & ((1u << lane) - 1u))] = s.p0 + 32 * (w - lane + k) + lane;
        }
        n0 += total;
        w0 += kWarps * each;
    }
    if (s.ranks > 1)
        meet(s.ranks);                                           // (nobody leaves while it is read)
}

// A cluster a (query token, kv head): its CTAs share out the tiles, work their scores
// out, which stay in shared memory, and select together.  Lengths and block tables may
// be read ahead of the kernel before, as by the decode; bounds and queries may not.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 1 : 2) page_select_kernel(const __grid_constant__ SelectParams p)
{
    extern __shared__ __align__(128) uint8_t ssmem[];
    __shared__ PickShared sh;
    constexpr int kWarps = kThreads / 32;
    uint4 *frag = reinterpret_cast<uint4 *>(ssmem + kWarps * kStages * kStageBytes);      // [kQueryWords]
    // page ids, and once a tile is worked on its scores
    uint32_t *place = reinterpret_cast<uint32_t *>(frag + kQueryWords);
    uint32_t *taken = place + p.chunk_tiles * kTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const long long unit = p.unit0 + blockIdx.x / ranks, row = unit / p.hkv;
    const int h = static_cast<int>(unit - row * p.hkv);
    const int b = static_cast<int>(row / p.q_len), t = static_cast<int>(row - static_cast<long long>(b) * p.q_len);
    const int len = __ldg(p.seq_lens + b), max_len = p.max_pages * kPageSize;
    if (h == 0 && t == 0 && rank == 0 && tid == 0 && (len < 0 || len > max_len))
        report(p.dev_status, NVFP4KV_DEV_BAD_LEN);
    const int pages = pages_seen(clamp_len(len, max_len), p.q_len, t);
    int32_t *out = p.pages + unit * p.budget;
    if (pages <= p.budget) {
        pdl_wait();
        for (int i = rank * kThreads + tid; i < p.budget; i += ranks * kThreads)
            out[i] = i < pages ? i : -1;
        return;
    }
    // this CTA's tiles (chunk_tiles at most) and pages
    const int all = (pages + kTile - 1) / kTile;
    const int begin = static_cast<int>(static_cast<long long>(all) * rank / ranks);
    const int tiles = static_cast<int>(static_cast<long long>(all) * (rank + 1) / ranks) - begin;
    const int p0 = begin * kTile, count = min(tiles * kTile, pages - p0);
    for (int i = tid; i < (tiles * kTile + 31) / 32; i += kThreads)
        taken[i] = 0;
    clear_counts<kThreads>(sh);
    if (tid == 0) {
        sh.least = 0xffffffffu;
        sh.most = 0;
    }
    const int32_t *table = p.block_table + static_cast<size_t>(b) * p.max_pages + p0;
    for (int i0 = tid; i0 < tiles * kTile; i0 += 8 * kThreads) {
        int phys[8];                                             // (asked for together)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            phys[k] = i0 + k * kThreads < count ? __ldg(table + i0 + k * kThreads) : 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i0 + k * kThreads < tiles * kTile)
                place[i0 + k * kThreads] = checked(p, phys[k]);
    }
    __syncthreads();
    pdl_wait();
    TileRing ring{smem_addr(ssmem) + warp * kStages * kStageBytes, {}};
#pragma unroll
    for (int k = 0; k < kStages; ++k) {
        const int tile = warp + k * kWarps;
        ring.ask(p, h, tile < tiles, tile < tiles ? place[tile * kTile + (lane & 15)] : 0, k, lane);
    }
    if (warp == kWarps - 1)
        load_queries(p, b, t, h, frag, lane);
    __syncthreads();
    // (read from shared memory for every tile, the queries would take as much of its
    // bandwidth as the tiles)
    uint4 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = frag[i * 32 + lane];
    const float2 from = reinterpret_cast<const float2 *>(frag + 8 * 32)[lane & 3];
    const int lo = max(p.first - p0, 0), hi = min(pages - p.last - p0, count);
    uint32_t least = 0xffffffffu, most = 0;
    for (int tile = warp; tile < tiles;) {
#pragma unroll
        for (int k = 0; k < kStages; ++k) {
            if (tile >= tiles)
                break;
            ring.wait();
            uint4 a[2][4];
            ring.read(k, a, lane);
            const float step = ring.step[k];
            const int next = tile + kStages * kWarps;
            ring.ask(p, h, next < tiles, next < tiles ? place[next * kTile + (lane & 15)] : 0, k, lane);
            const float score = score_of(a, [&](int i) { return w[i]; }, from, step, lane);
            const int i = tile * kTile + (lane & 15);
            if (lane < 16)
                place[i] = __float_as_uint(score);
            if (i >= lo && i < hi) {
                least = min(least, order_of(score));
                most = max(most, order_of(score));
            }
            tile += kWarps;
        }
    }
    __syncthreads();
    const Selection s{reinterpret_cast<const float *>(place), taken, p0, count, lo, hi, pages, p.first, p.last, rank, ranks};
    pick_pages<kThreads>(s, least, most, p.budget - p.first - p.last, out, sh);
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

// PickShared in a CTA's shared memory, in front of the dynamic part's 128-byte places.
constexpr int kPickStatic = (sizeof(PickShared) + 127) / 128 * 128;
// Dynamic shared memory that a launch may take, beside PickShared.
constexpr size_t kMostShared = 227 * 1024 - sizeof(PickShared) - 1024;

template <int kThreads>
static cudaError_t allow_select()
{
    return allow_shared<page_select_kernel<kThreads>, kPickStatic>();
}

template <int kThreads>
static cudaError_t launch_select(const SelectParams &p, long long units, size_t smem, int ranks, cudaStream_t s)
{
    const cudaError_t e = allow_select<kThreads>();
    if (e != cudaSuccess)
        return e;
    return launch_cluster(page_select_kernel<kThreads>, dim3(static_cast<unsigned>(units * ranks)), dim3(kThreads), ranks,
                          smem, s, p);
}

// Dynamic shared memory of a CTA with so many tiles.
static size_t select_bytes(int threads, int tiles)
{
    const size_t pages = static_cast<size_t>(tiles) * kTile;
    return threads / 32 * kStages * kStageBytes + kQueryWords * sizeof(uint4) + pages * 4 + (pages + 31) / 32 * 4;
}

// Whether two CTAs of 256 threads with all pages of a unit fit on an SM (1 KB of each is
// the system's): up to 5,136 pages.
static bool two_on_an_sm(int max_pages)
{
    return 2 * (select_bytes(256, (max_pages + kTile - 1) / kTile) + kPickStatic + 1024) <= 228 * 1024;
}

// CTAs of 512 threads, one an SM, or of 256, two an SM, and how many a cluster.  A
// meeting of the cluster costs a microsecond, which r CTAs repay from some 512 r^2
// pages on (8 heads of one sequence: 2,048 pages 12.6 us with one, 12.1 with two, 12.9
// with four; 4,096 pages 16.0 with two, 14.8 with three, 15.2 with four; 8,192 pages
// 23.7, 20.0, 19.3), as long as all clusters run at a time (48 units of 8,192 pages: 28
// us by clusters of two, 45 by 48 of three, whose last ones wait; 96 of 2,000: 15 and
// 27).  Where there are more units than SMs, two CTAs at a time on an SM work beside
// each other (560 units of 2,000 pages: 73 us with 512 threads, 62 with 256; 320 of
// 4,000: 84.2 and 83.5), as long as two fit: one alone has half the warps and loads in
// flight (160 units of 5,152 pages over the bounds of 24,000: 43 us with 512 threads, 59
// with 256; 560 of 8,125 over 84,000: 167 and 237).
static cudaError_t launch_units(const SelectParams &p, long long unit0, long long units, cudaStream_t s)
{
    const int tiles = (p.max_pages + kTile - 1) / kTile;
    const int threads = units > sm_count() && two_on_an_sm(p.max_pages) ? 256 : 512;
    int ranks = 1;
    if (units * 2 <= sm_count()) {
        while (ranks < 8 && (2 * ranks + 1) * (2 * ranks + 1) * 128 <= p.max_pages)
            ++ranks;                                             // (the next whole number to sqrt(pages / 512))
        const cudaError_t e = allow_select<512>();
        if (e != cudaSuccess)
            return e;
        while (ranks > 1 && units > clusters_at_once<page_select_kernel<512>, 512>(ranks, kMostShared))
            --ranks;
    }
    SelectParams q = p;
    q.unit0 = unit0;
    auto bytes = [&]() {
        q.chunk_tiles = (tiles + ranks - 1) / ranks;
        return select_bytes(threads, q.chunk_tiles);
    };
    static_assert(512 / 32 * kStages * kStageBytes + kQueryWords * sizeof(uint4) +
                          NVFP4KV_MAX_SELECT_PAGES / 8 / 8 * 33 + 1024 <= kMostShared, "the largest call fits eight CTAs");
    while (bytes() > kMostShared && ranks < 8)
        ++ranks;
    const size_t smem = bytes();
    return threads == 256 ? launch_select<256>(q, units, smem, ranks, s)
                          : launch_select<512>(q, units, smem, ranks, s);
}

// The units past the last full wave go by a launch of their own where they are few
// enough for clusters: 160 units of 8,125 pages in 78 us instead of 96, 192 in 82 instead
// of 97, 320 of 4,000 in 76 instead of 87, of 2,048 in 47.5 instead of 49.3.
cudaError_t launch_select_pages(const SelectParams &p, cudaStream_t s)
{
    const long long units = static_cast<long long>(p.batch) * p.q_len * p.hkv, sms = max(1, sm_count());
    const long long wave = units > sms && two_on_an_sm(p.max_pages) ? 2 * sms : sms;
    const long long full = p.max_pages >= 2048 ? units / wave * wave : 0;
    const long long rest = units - full;
    if (full == 0 || rest * 2 > sms || rest == 0)
        return launch_units(p, 0, units, s);
    const cudaError_t e = launch_units(p, 0, full, s);
    return e != cudaSuccess ? e : launch_units(p, full, rest, s);
}

} // namespace nvfp4kv
