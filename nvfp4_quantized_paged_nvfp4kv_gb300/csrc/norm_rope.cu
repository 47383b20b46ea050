// Head norm and position rotation of new queries and keys, alone or fused
// with the NVFP4 write of the keys and values.
//
// For a row x of 128 channels of one token and head, at position n:
//   y = x * rsqrt(mean_c x_c^2 + eps) * w        (w absent: y = x)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin),  angle n * f_i,
// for each of the R / 2 channel pairs (a, b): (i, i + R/2), or (2i, 2i + 1)
// when interleaved; channels from R on keep y.  All in fp32, rounded once to
// the output type.
//
// Angles.  n * f_i in fp32 is off by |angle| 2^-24: 0.06 radians at a position
// of a million.  f_i / 2 pi is kept as a 64-bit binary fraction of a turn
// instead, and n times it, modulo 2^64 as integers multiply, is the fraction
// of a turn exactly (up to n 2^-65); cos and sin are taken of its signed top
// 32 bits.
//
// Work split.  A row is eight lanes with 16 channels each (one cache block),
// so a warp instruction covers four heads of one token: the sum of squares is
// three shuffles, a half-split pair's partner is the same place in another
// lane of the row, and a lane holds a whole block for the quantiser.  A warp
// job is one token and a run of its heads: the job's cos and sin, multiplied
// by the weights of their channels, stay in 32 registers of the lane for all
// its heads.  Q jobs, K jobs and (fused) V blocks share one launch.
#include "nvfp4kv.h"
#include "record_write.cuh"

namespace nvfp4kv {
namespace {

constexpr int kNrThreads = 128;
constexpr int kNrWarps = kNrThreads / 32;

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi)
{
    const __nv_bfloat162 two = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&two);
}

// Sixteen channels of an input row to fp32.
template <bool kBf16>
__device__ __forceinline__ void store16(void *dst, size_t elem_off, const float (&y)[16])
{
    if constexpr (kBf16) {
        uint4 *d = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst) + elem_off);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            d[k] = make_uint4(bf16x2_bits(y[8 * k], y[8 * k + 1]), bf16x2_bits(y[8 * k + 2], y[8 * k + 3]),
                              bf16x2_bits(y[8 * k + 4], y[8 * k + 5]), bf16x2_bits(y[8 * k + 6], y[8 * k + 7]));
    } else {
        float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(dst) + elem_off);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            d[k] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
    }
}

// Plain (coherent) loads: an output row may be the input row.
template <bool kBf16>
__device__ __forceinline__ void load_row(const void *src, size_t elem_off, RawBlock<kBf16> &r)
{
    const uint4 *p = kBf16 ? reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + elem_off)
                           : reinterpret_cast<const uint4 *>(static_cast<const float *>(src) + elem_off);
#pragma unroll
    for (int i = 0; i < (kBf16 ? 2 : 4); ++i)
        r.v[i] = p[i];
}

__device__ __forceinline__ bool slot_site(const NormRopeParams &p, int slot, int h, size_t &record, int &tok,
                                          bool report_bad)
{
    if (slot < 0)
        return false;
    if (slot >= p.num_pages * kPageSize) {
        if (report_bad)
            report(p.dev_status, NVFP4KV_DEV_BAD_SLOT);
        return false;
    }
    const int page = slot / kPageSize;
    tok = slot - page * kPageSize;
    record = (static_cast<size_t>(page) * p.hkv + h) * kNvfp4Record;
    return true;
}

// Token t's rows head0 .. head0 + n - 1 of Q or K, by one warp.
template <bool kBf16, bool kAppend>
__device__ __forceinline__ void rows_job(const NormRopeParams &p, int t, int head0, int n, bool is_k, float2 *cs)
{
    const int lane = threadIdx.x & 31, part = lane & 7, sub = lane >> 3;
    const int pos = p.positions[t];
    if (pos < 0)
        return;                                  // a token that is not there: nothing is written
    const int half = p.rot >> 1;
    // the first rows' loads go out before the angles are worked out
    const void *src = is_k ? p.k : p.q;
    const size_t row = static_cast<size_t>(t) * (is_k ? p.k_stride : p.q_stride) + static_cast<size_t>(16 * part);
    RawBlock<kBf16> nxt;
    if (sub < n)
        load_row<kBf16>(src, row + static_cast<size_t>(head0 + sub) * kHeadDim, nxt);

    for (int i = lane; i < half; i += 32) {
        const uint64_t turn = p.freq[i] * static_cast<uint64_t>(pos);
        float sn, c;
        sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn, &c);
        cs[i] = make_float2(c * p.rope_scale, sn * p.rope_scale);
    }
    __syncwarp();
    // y_c = rstd (x_c wc + x_partner ws)
    const void *w = is_k ? p.k_weight : p.q_weight;
    auto weight = [&](int c) {
        if (w == nullptr)
            return 1.f;
        return p.weight_bf16 ? __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t *>(w) + c)) << 16)
                             : __ldg(static_cast<const float *>(w) + c);
    };
    float wc[16], ws[16];
    const int c0 = 16 * part;
    const bool turns = c0 < p.rot;
    int partner = part;
    if (turns && !p.interleaved)
        partner = c0 < half ? part + half / 16 : part - half / 16;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int c = c0 + j;
        const float wt = weight(c);
        wc[j] = wt;
        ws[j] = 0.f;
        if (turns) {
            if (p.interleaved) {
                const float2 a = cs[c >> 1];
                wc[j] = wt * a.x;
                ws[j] = (j & 1 ? a.y : -a.y) * weight(c ^ 1);
            } else {
                const bool low = c < half;
                const float2 a = cs[low ? c : c - half];
                wc[j] = wt * a.x;
                ws[j] = (low ? -a.y : a.y) * weight(low ? c + half : c - half);
            }
        }
    }
    const int from = (lane & 24) | partner;
    for (int r0 = 0; r0 < n; r0 += 4) {
        const bool live = r0 + sub < n;
        const RawBlock<kBf16> cur = nxt;
        if (r0 + 4 + sub < n)
            load_row<kBf16>(src, row + static_cast<size_t>(head0 + r0 + 4 + sub) * kHeadDim, nxt);
        float x[16], y[16];
        unpack<kBf16>(cur, x);
        float rstd = 1.f;
        if (w != nullptr) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j)
                sum = fmaf(x[j], x[j], sum);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                sum += __shfl_xor_sync(kFullMask, sum, o);
            rstd = rsqrtf(fmaf(sum, 1.f / kHeadDim, p.eps));
        }
        if (p.interleaved) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                y[j] = rstd * fmaf(x[j], wc[j], x[j ^ 1] * ws[j]);
        } else {
            RawBlock<kBf16> other;
#pragma unroll
            for (int i = 0; i < (kBf16 ? 2 : 4); ++i) {
                other.v[i].x = __shfl_sync(kFullMask, cur.v[i].x, from);
                other.v[i].y = __shfl_sync(kFullMask, cur.v[i].y, from);
                other.v[i].z = __shfl_sync(kFullMask, cur.v[i].z, from);
                other.v[i].w = __shfl_sync(kFullMask, cur.v[i].w, from);
            }
            float z[16];
            unpack<kBf16>(other, z);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                y[j] = rstd * fmaf(x[j], wc[j], z[j] * ws[j]);
        }
        if (!live)
            continue;
        const int head = head0 + r0 + sub;
        if (!is_k) {
            store16<true>(p.q_out, (static_cast<size_t>(t) * p.hq + head) * kHeadDim + c0, y);
        } else if constexpr (!kAppend) {
            store16<kBf16>(p.k_out, (static_cast<size_t>(t) * p.hkv + head) * kHeadDim + c0, y);
        } else {
            size_t rec;
            int tok;
            if (!slot_site(p, p.slot_mapping[t], head, rec, tok, head == 0 && part == 0))
                continue;
            // the cache holds what the key would be in the input type: the
            // same bytes as storing it and quantising the stored row
            if constexpr (kBf16) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    y[j] = __bfloat162float(__float2bfloat16_rn(y[j]));
            }
            const uint32_t flip = divide_by_tensor_scale(y, head_tensor_scale(p.hs, false, head, p.gscale));
            write_nvfp4_block(p.pool + rec, false, tok, part, y, ScaleOfByte(), flip);
        }
    }
}

// V block `blk` of head h for the pr-th token pair of the call (pairs begin
// one token early when the first slot is odd, so consecutive slots form the
// record's token pairs).
template <bool kBf16>
__device__ __forceinline__ void v_pair_job(const NormRopeParams &p, int pr, int h, int blk)
{
    const int first = p.slot_mapping[0];
    const int o = first >= 0 ? (first & 1) : 0;
    const int t0 = 2 * pr - o, t1 = t0 + 1;
    const bool has0 = t0 >= 0 && t0 < p.num_tokens, has1 = t1 < p.num_tokens;
    const size_t off = static_cast<size_t>(h) * kHeadDim + blk * 16;
    RawBlock<kBf16> r0, r1;
    if (has0)
        load_row<kBf16>(p.v, static_cast<size_t>(t0) * p.v_stride + off, r0);
    if (has1)
        load_row<kBf16>(p.v, static_cast<size_t>(t1) * p.v_stride + off, r1);
    const int s0 = has0 && p.positions[t0] >= 0 ? p.slot_mapping[t0] : -1;
    const int s1 = has1 && p.positions[t1] >= 0 ? p.slot_mapping[t1] : -1;
    size_t rec0 = 0, rec1 = 0;
    int tok0 = 0, tok1 = 0;
    const bool ok0 = slot_site(p, s0, h, rec0, tok0, false);
    const bool ok1 = slot_site(p, s1, h, rec1, tok1, false);
    const TensorScale G = tensor_scale(head_tensor_scale(p.hs, true, h, p.gscale));
    float x[16];
    if (ok0 && ok1 && (s0 & 1) == 0 && s1 == s0 + 1) {
        uint32_t S0, S1, q0[2], q1[2];
        unpack<kBf16>(r0, x);
        uint32_t flip = divide_by_tensor_scale(x, G);
        quantize_block(x, S0, q0, ScaleOfByte(), flip);
        unpack<kBf16>(r1, x);
        flip = divide_by_tensor_scale(x, G);
        quantize_block(x, S1, q1, ScaleOfByte(), flip);
        write_nvfp4_v_pair(p.pool + rec0, tok0, blk, S0, q0, S1, q1);
        return;
    }
    if (ok0) {
        unpack<kBf16>(r0, x);
        const uint32_t flip = divide_by_tensor_scale(x, G);
        write_nvfp4_block(p.pool + rec0, true, tok0, blk, x, ScaleOfByte(), flip);
    }
    if (ok1) {
        unpack<kBf16>(r1, x);
        const uint32_t flip = divide_by_tensor_scale(x, G);
        write_nvfp4_block(p.pool + rec1, true, tok1, blk, x, ScaleOfByte(), flip);
    }
}

// Warp jobs, token-major: per token q_jobs runs of Q heads and k_jobs runs of
// K heads; then the V blocks, one a thread.
template <bool kBf16, bool kAppend>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p)
{
    __shared__ float2 cs[kNrWarps][kHeadDim / 2];
    // (the wait comes before the trigger: a kernel that starts early behind
    // this one finds everything before it complete)
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const long long job = static_cast<long long>(blockIdx.x) * kNrWarps + warp;
    const int per = p.q_jobs + p.k_jobs;
    const long long row_jobs = static_cast<long long>(p.num_tokens) * per;
    if (job < row_jobs) {
        const int t = static_cast<int>(job / per);
        int j = static_cast<int>(job - static_cast<long long>(t) * per);
        const bool is_k = j >= p.q_jobs;
        if (is_k)
            j -= p.q_jobs;
        const int heads = is_k ? p.hkv : p.hq;
        const int head0 = j * p.heads_per_job;
        rows_job<kBf16, kAppend>(p, t, head0, min(p.heads_per_job, heads - head0), is_k, cs[warp]);
    } else if constexpr (kAppend) {
        const long long item = (job - row_jobs) * 32 + (threadIdx.x & 31);
        const long long unit = item >> 3;        // pair * hkv + h
        const long long pr = unit / p.hkv;
        if (2 * pr <= p.num_tokens)              // (the early start adds half a pair)
            v_pair_job<kBf16>(p, static_cast<int>(pr), static_cast<int>(unit - pr * p.hkv),
                              static_cast<int>(item & 7));
    }
}

} // namespace

cudaError_t launch_norm_rope(const NormRopeParams &in, cudaStream_t s)
{
    NormRopeParams p = in;
    // four heads a job while that leaves fewer jobs than fill the SMs twice
    // over, else sixteen, so a job's angles serve more rows
    const long long quads = static_cast<long long>(p.num_tokens) * ((p.hq + 3) / 4 + (p.hkv + 3) / 4);
    p.heads_per_job = quads < 32LL * sm_count() ? 4 : 16;
    p.q_jobs = (p.hq + p.heads_per_job - 1) / p.heads_per_job;
    p.k_jobs = (p.hkv + p.heads_per_job - 1) / p.heads_per_job;
    long long warps = static_cast<long long>(p.num_tokens) * (p.q_jobs + p.k_jobs);
    const bool append = p.pool != nullptr;
    if (append)
        warps += ((static_cast<long long>(p.num_tokens) + 2) / 2 * p.hkv * 8 + 31) / 32;
    const long long grid = (warps + kNrWarps - 1) / kNrWarps;
    if (grid > 0x7fffffffLL)
        return cudaErrorInvalidValue;
    const auto kernel = append ? (p.in_bf16 ? norm_rope_kernel<true, true> : norm_rope_kernel<false, true>)
                               : (p.in_bf16 ? norm_rope_kernel<true, false> : norm_rope_kernel<false, false>);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kNrThreads), 0, s, p);
}

} // namespace nvfp4kv
