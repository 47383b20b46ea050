// The block-scaled FP8 cache: new rows written, cached rows read back.
//
// A block is one page of one kv head, K and V apart: 16 tokens x 128 channels
// that share a scale s = 2^e, e the least integer with amax <= 448 * 2^e (from
// -100 to 100), code = E4M3_rn(x / s).  A page is filled over several calls:
// the scale of a page that holds tokens already rises where new ones need it
// (s = max(s_old, s(new))), and the codes that are there are rounded anew,
// E4M3_rn(code * s_old / s).  That is why scales are powers of two: x / s is
// exact, and so is the new rounding but for codes that become subnormal, so a
// page filled token by token holds what the same tokens written at once hold
// but for those (with amax / 448 for a scale every rise would round all of the
// page again).  A page whose first token comes with the call starts afresh.
#include "decode_common.cuh"

namespace nvfp4kv {
namespace {

constexpr int kLeastExp = -100, kMostExp = 100;

__device__ __forceinline__ float two_to(int e)
{
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Least e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), within the limits.
__device__ __forceinline__ int scale_exp(float amax)
{
    const uint32_t bits = __float_as_uint(amax) & 0x7fffffffu;
    const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
    return max(kLeastExp, min(kMostExp, e));
}

// Eight channels of a row, as fp32.
template <bool kBf16>
struct Eight {
    uint4 v[kBf16 ? 1 : 2];

    __device__ __forceinline__ void load(const void *src, size_t elem)
    {
        const uint4 *p = kBf16 ? reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + elem)
                               : reinterpret_cast<const uint4 *>(static_cast<const float *>(src) + elem);
#pragma unroll
        for (int i = 0; i < (kBf16 ? 1 : 2); ++i)
            v[i] = p[i];
    }

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (kBf16 ? 1 : 2); ++i)
            v[i] = make_uint4(0, 0, 0, 0);
    }

    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kBf16) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
        if constexpr (!kBf16) {
            const uint32_t z[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[4 + i] = __uint_as_float(z[i]);
        }
    }
};

// Eight E4M3 codes (two words, channel order) of x * by.
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float by)
{
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = f32x2_to_e4m3x2(x[2 * i] * by, x[2 * i + 1] * by);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// The codes times `by`, rounded anew.
__device__ __forceinline__ uint2 recode(uint2 c, float by)
{
    float x[8];
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t a, b;
        e4m3x4_to_f16x2x2(w[i], a, b);
        const float2 fa = __half22float2(*reinterpret_cast<__half2 *>(&a));
        const float2 fb = __half22float2(*reinterpret_cast<__half2 *>(&b));
        x[4 * i] = fa.x;
        x[4 * i + 1] = fa.y;
        x[4 * i + 2] = fb.x;
        x[4 * i + 3] = fb.y;
    }
    return codes_of(x, by);
}

// Whether rows c0 .. c1 - 1 can be the last ones of a sequence of len tokens.
__device__ __forceinline__ bool good_range(const BlockAppendParams &p, int c0, int c1, int len)
{
    return c0 >= 0 && c1 >= c0 && c1 <= p.num_tokens && len >= c1 - c0 && len <= p.max_pages * kPageSize;
}

// Last sequence whose first unit is at or before u, by the whole warp (32
// probes a round); -1 where there is none.  Sequence b's units begin at
// floor(q_indptr[b] / 16) + 2b: its pages are at most floor(C / 16) + 2.
__device__ __forceinline__ int find_unit(const int32_t *q_indptr, int batch, long long u, int lane)
{
    int lo = 0, hi = batch;
    for (;;) {
        const int step = (hi - lo + 31) / 32, at = lo + step * lane;
        const bool below = at < hi && (static_cast<long long>(__ldg(q_indptr + min(at, batch - 1))) >> 4) + 2 * at <= u;
        const int n = __popc(__ballot_sync(kFullMask, below));
        if (n == 0)
            return -1;
        lo += step * (n - 1);
        hi = min(hi, lo + step);
        if (step == 1)
            return lo;
    }
}

// One warp a (page, kv head, K or V).  A half warp holds a pair of tokens (2p,
// 2p + 1) at a time, lane c of it channels 8c .. 8c + 7 of both: 16 bytes a
// load of bf16, whole rows a half warp, and a V record's 16-byte chunk (the two
// tokens' bytes interleaved) is one lane's.  All rows of the page are asked for
// before the first is used; the page's old codes and scale come beside them.
// Three prompts, 12,288 rows of 8 heads in bf16: 16.6 us for 75 MB, two thirds of the
// copy rate, bound by the latency of its one round of loads (24 warps an SM; K and V in
// one warp, with twice the registers, 20.6 us; more warps of fewer rows: no faster).
template <bool kBf16>
__global__ void __launch_bounds__(256, kBf16 ? 3 : 2) block_append_kernel(const __grid_constant__ BlockAppendParams p)
{
    pdl_wait();                  // the records may still be read, the tables still be written
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long id = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
    const long long u = id / (2 * p.hkv);
    const int hv = static_cast<int>(id - u * 2 * p.hkv), h = hv >> 1;
    const bool is_v = hv & 1;
    // The ranges are reported on by the first warps, a lane a sequence (there are at
    // least 4 warps a sequence): one that points outside the rows may own no unit here.
    if (id * 32 < p.batch) {
        const int mine = static_cast<int>(id) * 32 + lane;
        if (mine < p.batch && !good_range(p, __ldg(p.q_indptr + mine), __ldg(p.q_indptr + mine + 1), __ldg(p.seq_lens + mine)))
            report(p.dev_status, NVFP4KV_DEV_BAD_LEN);
    }
    const int b = find_unit(p.q_indptr, p.batch, u, lane);
    if (b < 0)
        return;
    const int c0 = __ldg(p.q_indptr + b), c1 = __ldg(p.q_indptr + b + 1), len = __ldg(p.seq_lens + b);
    const long long i = u - ((static_cast<long long>(c0) >> 4) + 2 * b);     // page of the sequence's new ones
    if (!good_range(p, c0, c1, len))
        return;
    const int pos0 = len - (c1 - c0);
    const long long page = pos0 / kPageSize + i;
    const int begin = static_cast<int>(max(static_cast<long long>(pos0), page * kPageSize) - page * kPageSize);
    const long long rest = len - page * kPageSize;
    const int end = static_cast<int>(rest < kPageSize ? rest : kPageSize);   // tokens begin .. end - 1 are new
    if (begin >= end)
        return;
    const int phys = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + page);
    if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_pages)) {
        if (hv == 0 && lane == 0)
            report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);
        return;
    }
    uint8_t *rec = p.pool + (static_cast<size_t>(phys) * p.hkv + h) * kFp8BlockRecord;
    float *scale = reinterpret_cast<float *>(rec + kFp8Record) + is_v;
    const void *src = is_v ? p.v_new : p.k_new;
    const int half = lane >> 4, c = lane & 15;
    const long long row0 = c0 + page * kPageSize - pos0;                     // row of the page's token 0

    Eight<kBf16> x[4][2];
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int t0 = 4 * it + 2 * half;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (t0 + w >= begin && t0 + w < end)
                x[it][w].load(src, (static_cast<size_t>(row0 + t0 + w) * p.hkv + h) * kHeadDim + 8 * c);
            else
                x[it][w].zero();
        }
    }
    int e_old = kLeastExp;
    if (begin > 0) {
        e_old = max(kLeastExp, min(kMostExp, static_cast<int>((__float_as_uint(__ldcg(scale)) >> 23) & 0xffu) - 127));
        // the codes that are there, into L2: they are wanted if the scale rises, V's
        // of a shared pair in any case
        asm volatile("prefetch.global.L2 [%0];" ::"l"(rec + (is_v ? 2048 : 0) + 64 * lane));
    }
    float amax = 0.f;
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float f[8];
            x[it][w].get(f);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                amax = fmaxf(amax, fabsf(f[k]));
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
    const int e = max(e_old, scale_exp(amax));
    const float by = two_to(-e);
    const bool raised = begin > 0 && e > e_old;
    const int shift = e_old - e;                             // 2^shift: at most 1, from 2^-126 on as good as 0
    const float down = shift < -126 ? 0.f : two_to(shift);
    __syncwarp();                // (the old scale has been read)
    if (lane == 0 && (begin == 0 || raised))
        *scale = two_to(e);

#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int pr = 2 * it + half, t0 = 2 * pr;
        if (t0 >= end || (t0 + 1 < begin && !raised))
            continue;                                        // nothing of the pair is written
        uint2 code[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float f[8];
            x[it][w].get(f);
            code[w] = codes_of(f, by);
        }
        if (is_v) {
            const int f = (pr & 1) + 4 * ((pr >> 1) & 1);
            uint4 *at = reinterpret_cast<uint4 *>(rec + 2048 + pr * 256 + ((c + f) & 15) * 16);
            if (t0 < begin) {
                // byte 2i + w of the chunk is token w's channel i
                const uint4 o = __ldcg(at);
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    if (t0 + w < begin) {
                        code[w] = make_uint2(__byte_perm(o.x, o.y, w ? 0x7531 : 0x6420),
                                             __byte_perm(o.z, o.w, w ? 0x7531 : 0x6420));
                        if (raised)
                            code[w] = recode(code[w], down);
                    }
            }
            *at = make_uint4(__byte_perm(code[0].x, code[1].x, 0x5140), __byte_perm(code[0].x, code[1].x, 0x7362),
                             __byte_perm(code[0].y, code[1].y, 0x5140), __byte_perm(code[0].y, code[1].y, 0x7362));
        } else {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                uint2 *at = reinterpret_cast<uint2 *>(rec + (t0 + w) * 128 + (((c >> 1) + w) & 7) * 16 + (c & 1) * 8);
                if (t0 + w >= begin) {
                    if (t0 + w < end)
                        *at = code[w];
                } else if (raised) {
                    *at = recode(__ldcg(at), down);
                }
            }
        }
    }
}

// ---- reading back ------------------------------------------------------------

// Eight values of two words of codes to out (element offset `at`).
template <int kType>
__device__ __forceinline__ void put_eight(void *out, size_t at, uint2 c, float s)
{
    float x[8];
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t a, b;
        e4m3x4_to_f16x2x2(w[i], a, b);
        const float2 fa = __half22float2(*reinterpret_cast<__half2 *>(&a));
        const float2 fb = __half22float2(*reinterpret_cast<__half2 *>(&b));
        x[4 * i] = fa.x * s;
        x[4 * i + 1] = fa.y * s;
        x[4 * i + 2] = fb.x * s;
        x[4 * i + 3] = fb.y * s;
    }
    if constexpr (kType == NVFP4KV_F32) {
        float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else if constexpr (kType == NVFP4KV_BF16) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            h[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = f32x2_to_e4m3x2(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(out) + at) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    }
}

constexpr int kReadThreads = 256;

// One warp a page's K or V of one kv head: 16 lanes a row, eight channels a lane,
// so that a half warp writes whole rows of one head.  The same 12,288 rows: 14.5 us for
// 75 MB, two of three bytes written (K and V in one warp 18.1; other grids: the same).
template <int kType>
__global__ void __launch_bounds__(kReadThreads, 5) block_read_kernel(const __grid_constant__ BlockReadParams p)
{
    extern __shared__ int32_t rsmem[];
    int32_t *scratch = rsmem, *prefix = rsmem + kPrefixScratch;
    pdl_wait();
    pdl_launch_dependents();
    build_prefix(p.lens, p.batch, 1, p.max_pages * kPageSize, prefix, scratch, blockIdx.x == 0 ? p.dev_status : nullptr);
    const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
    const unsigned both = 2u * p.hkv;
    const long long units = static_cast<long long>(prefix[p.batch]) * both;
    const long long step = static_cast<long long>(gridDim.x) * (kReadThreads / 32);
    for (long long u = static_cast<long long>(blockIdx.x) * (kReadThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
        const int pg = units < (1LL << 32) ? static_cast<int>(static_cast<unsigned>(u) / both) : static_cast<int>(u / both);
        const int hv = static_cast<int>(u - static_cast<long long>(pg) * both), h = hv >> 1;
        const bool is_v = hv & 1;
        const int b = find_seq(prefix, p.batch, pg);
        const int page = pg - prefix[b];
        const int len = min(__ldg(p.lens + b), p.max_pages * kPageSize);
        int phys = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + page);
        const long long row = static_cast<long long>(__ldg(p.kv_indptr + b)) + page * kPageSize;
        if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_pages)) {
            if (hv == 0 && lane == 0)
                report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);
            phys = 0;
        }
        const uint8_t *rec = p.pool + (static_cast<size_t>(phys) * p.hkv + h) * kFp8BlockRecord;
        const float s = reinterpret_cast<const float *>(rec + kFp8Record)[is_v];
        const int valid = len - page * kPageSize;
        void *out = is_v ? p.v_out : p.k_out;
        // a row's place: channels 8c .. of token t at row t
        const size_t at = (static_cast<size_t>(row) * p.hkv + h) * kHeadDim + 8 * c, next = static_cast<size_t>(p.hkv) * kHeadDim;
        if (!is_v) {
            uint2 x[8];                                          // tokens 2i + half
            const uint2 *src = reinterpret_cast<const uint2 *>(rec) + 16 * half + 2 * (((c >> 1) + half) & 7) + (c & 1);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = src[32 * i];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (2 * i + half < valid)
                    put_eight<kType>(out, at + (2 * i + half) * next, x[i], s);
        } else {
            uint4 x[4];                                          // token pairs 2i + half
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pr = 2 * i + half, f = (pr & 1) + 4 * ((pr >> 1) & 1);
                x[i] = reinterpret_cast<const uint4 *>(rec + 2048)[16 * pr + ((c + f) & 15)];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int t = 2 * (2 * i + half) + w;
                    if (t < valid)
                        put_eight<kType>(out, at + t * next,
                                         make_uint2(__byte_perm(x[i].x, x[i].y, w ? 0x7531 : 0x6420),
                                                    __byte_perm(x[i].z, x[i].w, w ? 0x7531 : 0x6420)),
                                         s);
                }
        }
    }
}

template <int kType>
cudaError_t launch_read(const BlockReadParams &p, cudaStream_t s)
{
    const size_t smem = (kPrefixScratch + static_cast<size_t>(p.batch) + 1) * sizeof(int32_t);
    const long long warps = static_cast<long long>(p.batch) * p.max_pages * p.hkv * 2;
    long long grid = static_cast<long long>(sm_count()) * 6;
    grid = min(grid, (warps + kReadThreads / 32 - 1) / (kReadThreads / 32));
    return launch_pdl(block_read_kernel<kType>, dim3(static_cast<unsigned>(grid)), dim3(kReadThreads), smem, s, p);
}

} // namespace

cudaError_t launch_block_append(const BlockAppendParams &p, cudaStream_t s)
{
    const long long units = static_cast<long long>(p.num_tokens) / kPageSize + 2LL * p.batch;
    const long long grid = (units * p.hkv * 2 + 7) / 8;
    if (grid > 0x7fffffffLL)
        return cudaErrorInvalidValue;
    return launch_pdl(p.in_bf16 ? block_append_kernel<true> : block_append_kernel<false>,
                      dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, p);
}

cudaError_t launch_block_read(const BlockReadParams &p, cudaStream_t s)
{
    switch (p.out_dtype) {
    case NVFP4KV_F32:
        return launch_read<NVFP4KV_F32>(p, s);
    case NVFP4KV_BF16:
        return launch_read<NVFP4KV_BF16>(p, s);
    default:
        return launch_read<NVFP4KV_E4M3>(p, s);
    }
}

} // namespace nvfp4kv
