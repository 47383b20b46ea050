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
// of a turn to n 2^-63 (f_i / 2 pi is cut to 64 bits in two parts); cos and sin
// are taken of its signed top 32 bits.
//
// Work split.  A row is eight lanes, lane l with channels 8l .. 8l + 7 and 64 +
// 8l .. 64 + 8l + 7, so that eight lanes load or store 128 bytes on end (16
// channels on end a lane touched every 32-byte sector twice: 63 us for 8,192
// tokens of 48 + 8 heads, 43 now), a warp instruction covers four heads of one
// token (a quad), and the half-split partner of a full rotation is in the lane
// itself.  A token's quads are its queries', then its keys'; each warp takes an
// equal run of the call's quads (whole tokens, 2.7 a warp, left a tenth of the
// warps' time idle).  A token's cos and sin, multiplied by the weights of their
// channels, are worked out once by the warp (each lane doing so for its own 16
// channels cost 15 us) and stay in 32 registers of the lane for all its heads of
// a kind; products run on packed fp32 pairs.  For the cache two neighbouring
// lanes swap halves and hold a whole 16-value block each.  The rows and (fused)
// the V blocks share one launch of resident CTAs.
//
// Loads.  Four heads are 1 KB on end (2 KB in fp32); each warp keeps a ring of
// them in shared memory, filled by bulk copies that run ahead of the work and
// across its tokens.
//
// Bound.  8,192 bf16 tokens of 48 + 8 heads out of a fused projection's rows:
// 235 MB in 43 us, 5.5 TB/s, 82% of a copy's rate, with 56% of the issue slots
// taken.  With the cache write, 244 MB in 43 us.
#include "nvfp4kv.h"
#include "record_write.cuh"
#include <type_traits>

namespace nvfp4kv {
namespace {

constexpr int kNrThreads = 128;
constexpr int kNrWarps = kNrThreads / 32;

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi)
{
    const __nv_bfloat162 two = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&two);
}

// A lane's two pieces of an output row, the first at dst.
template <bool kBf16>
__device__ __forceinline__ void store_pieces(uint8_t *dst, const float (&y)[16])
{
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float *v = y + 8 * k;
        if constexpr (kBf16)
            *reinterpret_cast<uint4 *>(dst + 128 * k) =
                make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]),
                           bf16x2_bits(v[6], v[7]));
        else {
            float4 *d = reinterpret_cast<float4 *>(dst + 256 * k);
            d[0] = make_float4(v[0], v[1], v[2], v[3]);
            d[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
}

// A lane's two pieces of a row staged at `row`.
template <bool kBf16>
__device__ __forceinline__ void read_pieces(uint32_t row, int part, RawBlock<kBf16> &r)
{
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if constexpr (kBf16) {
            r.v[k] = lds128(row + 16 * part + 128 * k);
        } else {
            r.v[2 * k] = lds128(row + 32 * part + 256 * k);
            r.v[2 * k + 1] = lds128(row + 32 * part + 256 * k + 16);
        }
    }
}

// Sixteen values on end.
template <bool kBf16>
__device__ __forceinline__ void load_row(const void *src, size_t elem_off, RawBlock<kBf16> &r)
{
    const uint4 *p = kBf16 ? reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + elem_off)
                           : reinterpret_cast<const uint4 *>(static_cast<const float *>(src) + elem_off);
#pragma unroll
    for (int i = 0; i < (kBf16 ? 2 : 4); ++i)
        r.v[i] = p[i];
}

__device__ __forceinline__ uint4 shuffled(const uint4 &v, int from)
{
    return make_uint4(__shfl_sync(kFullMask, v.x, from), __shfl_sync(kFullMask, v.y, from),
                      __shfl_sync(kFullMask, v.z, from), __shfl_sync(kFullMask, v.w, from));
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

template <bool kBf16>
struct Ring {
    static constexpr int kStages = 4;                        // quads in flight a warp
    static constexpr uint32_t kRow = kHeadDim * (kBf16 ? 2 : 4);
    static constexpr uint32_t kStage = 4 * kRow;
    static constexpr int kCtas = kBf16 ? 5 : 4;              // on an SM (registers)
    static constexpr uint32_t kSmem = kNrWarps * kStages * kStage;
    static_assert(kCtas * (kSmem + 4608) <= 227 * 1024, "shared memory");
};

// What a CTA keeps in shared memory beside the rings: the weights of both kinds
// as fp32, the frequencies, each warp's angles, its rotation tables (of two
// channels 2u, 2u + 1 at a place: cos times weight, and the signed sin times the
// partner's weight) and its ring's barriers.
struct NrShared {
    float weight[2][kHeadDim];
    uint64_t freq[kHeadDim / 2];
    float2 cs[kNrWarps][kHeadDim / 2];
    float4 table[kNrWarps][kHeadDim / 2];
    uint64_t bar[kNrWarps][Ring<true>::kStages];
};

// The copies of a warp's quads, one after the other: `left` to go, the next one's
// rows at src, `heads` of its kind and token from there on.
template <bool kBf16>
struct Feed {
    const uint8_t *src;
    int t, left, heads;
    bool is_k;

    // head `head` of token t
    __device__ __forceinline__ void at(const NormRopeParams &p, int head)
    {
        const size_t elem = static_cast<size_t>(t) * (is_k ? p.k_stride : p.q_stride) + head * kHeadDim;
        src = static_cast<const uint8_t *>(is_k ? p.k : p.q) + elem * (kBf16 ? 2 : 4);
        heads = (is_k ? p.hkv : p.hq) - head;
    }
    __device__ __forceinline__ Feed(const NormRopeParams &p, int token, int quad, int n)
        : t(token), left(n), is_k(quad >= p.q_quads)
    {
        at(p, 4 * (is_k ? quad - p.q_quads : quad));
    }
    // the next quad to `stage` (whole warp; lane 0 copies)
    __device__ __forceinline__ void fetch(const NormRopeParams &p, uint32_t stage, uint32_t bar)
    {
        using G = Ring<kBf16>;
        if ((threadIdx.x & 31) == 0) {
            const uint32_t bytes = min(4, heads) * G::kRow;
            mbar_arrive_expect_tx(bar, bytes);
            bulk_g2s(stage, src, bytes, bar);
        }
        src += G::kStage;
        heads -= 4;
        if (--left > 0 && heads <= 0) {
            t += is_k;
            is_k = !is_k;
            at(p, 0);
        }
    }
};

// Where a channel's partner is: in the lane's other piece (half-split rotations of
// all channels), in the neighbouring channel (interleaved ones, and no rotation),
// or in another lane (half-split ones of some channels).  A kernel each: what the
// others need costs registers and instruction fetches (half-split, with the cache
// write: 43.1 us alone, 44.5 beside one other form, 46.0 beside two).
enum Pairs : int { kOpposite, kNeighbours, kTwoLanes };

// One warp's rows, quads from .. to - 1 of the call.  False when a wait for staged
// rows gave up.
template <bool kBf16, bool kAppend, int kPairs>
__device__ __forceinline__ bool rows_of_warp(const NormRopeParams &p, NrShared &sh, uint32_t ring, long long from,
                                             long long to)
{
    using G = Ring<kBf16>;
    const int lane = threadIdx.x & 31, part = lane & 7, sub = lane >> 3, warp = threadIdx.x >> 5;
    float2 *cs = sh.cs[warp];
    const uint32_t bar = smem_addr(sh.bar[warp]);
    const int half = p.rot >> 1;
    const int c0 = 8 * part;                     // channel of value j: c0 + (j & 7) + 64 (j / 8)

    int t = static_cast<int>(from / p.quads), quad = static_cast<int>(from - static_cast<long long>(t) * p.quads);
    int left = static_cast<int>(to - from);
    if (left <= 0)
        return true;
    Feed<kBf16> feed(p, t, quad, left);
    for (int st = 0; st < G::kStages && feed.left > 0; ++st)
        feed.fetch(p, ring + st * G::kStage, bar + 8 * st);

    uint32_t st = 0, phase = 0;
    int end = quad;
    bool ok = true;
    for (; ok && left > 0; ++t, quad = 0) {
    end = min(p.quads, quad + left);
    left -= end - quad;
    const int pos = p.positions[t];              // < 0: a token that is not there, nothing of it is written
    __syncwarp();                                // (the last token's angles have been read)
    for (int i = lane; i < half; i += 32) {
        const uint64_t turn = sh.freq[i] * static_cast<uint64_t>(static_cast<uint32_t>(max(pos, 0)));
        float sn, c;
        sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn, &c);
        cs[i] = make_float2(c * p.rope_scale, sn * p.rope_scale);
    }
    __syncwarp();
    // y_c = rstd (x_c wc + x_partner ws), two channels in a register.  A channel
    // that is not turned must not see any other one, whose infinity or NaN would
    // reach it through a zero factor.  It has -0 for ws and 0 for its partner (and
    // so keeps the sign of a zero), or, in bf16 rows whose pieces come by shuffles,
    // itself for its partner and half the weight for both: x w / 2, rounded, plus
    // x w / 2 rounds to what x w rounds to (2 us less than zeroing the pieces;
    // fp32 rows may hold values whose half is not a number of fp32).
    constexpr bool kHalves = kPairs == kTwoLanes && kBf16;
    uint64_t wc[8], ws[8];
    auto tables = [&](const float *wt) {
        float4 *tab = sh.table[warp];
        __syncwarp();                            // the last table has been read
#pragma unroll
        for (int u = lane; u < kHeadDim / 2; u += 32) {
            // place u: piece u / 32, channels 64 piece + 8 (u mod 8) + 2 (u / 8 mod 4) and the next
            const int c = 64 * (u >> 5) + 8 * (u & 7) + 2 * ((u >> 3) & 3);
            const float2 own = *reinterpret_cast<const float2 *>(wt + c);
            float4 v = kHalves ? make_float4(0.5f * own.x, 0.5f * own.y, 0.5f * own.x, 0.5f * own.y)
                               : make_float4(own.x, own.y, -0.f, -0.f);
            if (c < p.rot) {
                if (p.interleaved) {
                    const float2 a = cs[c >> 1];
                    v = make_float4(own.x * a.x, own.y * a.x, -a.y * own.y, a.y * own.x);
                } else {
                    const bool low = c < half;
                    const int mate = low ? c + half : c - half;
                    const float4 a = *reinterpret_cast<const float4 *>(cs + (low ? c : mate));
                    const float2 m = *reinterpret_cast<const float2 *>(wt + mate);
                    v = make_float4(own.x * a.x, own.y * a.z, (low ? -a.y : a.y) * m.x, (low ? -a.w : a.w) * m.y);
                }
            }
            tab[u] = v;
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 v = tab[32 * (j >> 2) + 8 * (j & 3) + part];
            wc[j] = f32x2_pack(v.x, v.y);
            ws[j] = f32x2_pack(v.z, v.w);
        }
    };
    // where a half-split partner piece is, when not in the lane itself: chunk
    // (of eight channels) 8 k + part of the row, plus or minus half / 8
    auto mate_chunk = [&](int k) {
        const int chunk = 8 * k + part;
        return 8 * chunk < half ? chunk + half / 8 : (8 * chunk < p.rot ? chunk - half / 8 : chunk);
    };
    while (ok && quad < end) {                   // the queries, then the keys
    const bool is_k = quad >= p.q_quads;
    const int stop = is_k ? end : min(end, p.q_quads);
    tables(sh.weight[is_k]);
    const bool normed = (is_k ? p.k_weight : p.q_weight) != nullptr;
    const int heads = is_k ? p.hkv : p.hq, head = 4 * (is_k ? quad - p.q_quads : quad) + sub;
    int ahead = pos >= 0 ? heads - head : 0;     // (positive: the lane's head is there)
    const size_t out_row = (static_cast<size_t>(t) * heads + head) * kHeadDim + c0;
    uint8_t *out = static_cast<uint8_t *>(is_k ? p.k_out : p.q_out) + out_row * (is_k && !kBf16 ? 4 : 2);
    for (; quad < stop; ++quad, ahead -= 4, out += 4 * kHeadDim * (is_k && !kBf16 ? 4 : 2)) {
        const bool live = ahead > 0;
        ok = __all_sync(kFullMask, mbar_wait_bounded(bar + 8 * st, phase, p.wait_limit));
        if (!ok)
            break;
        RawBlock<kBf16> cur;                     // (rows behind the last head: what the stage held, not written)
        read_pieces<kBf16>(ring + st * G::kStage + sub * G::kRow, part, cur);
        if (feed.left > 0) {
            fence_async_shared();                // the stage's reads before its next copy
            __syncwarp();
            feed.fetch(p, ring + st * G::kStage, bar + 8 * st);
        }
        if (++st == G::kStages) {
            st = 0;
            phase ^= 1u;
        }
        float x[16], y[16];
        unpack<kBf16>(cur, x);
        uint64_t x2[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x2[j] = f32x2_pack(x[2 * j], x[2 * j + 1]);
        uint64_t rstd2 = f32x2_pack(1.f, 1.f);
        if (normed) {
            uint64_t a = mul_f32x2(x2[0], x2[0]), b = mul_f32x2(x2[1], x2[1]);
#pragma unroll
            for (int j = 2; j < 8; j += 2) {
                a = fma_f32x2(x2[j], x2[j], a);
                b = fma_f32x2(x2[j + 1], x2[j + 1], b);
            }
            a = add_f32x2(a, b);
            float sum = f32x2_lo(a) + f32x2_hi(a);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                sum += __shfl_xor_sync(kFullMask, sum, o);
            const float rstd = rsqrtf(fmaf(sum, 1.f / kHeadDim, p.eps));
            rstd2 = f32x2_pack(rstd, rstd);
        }
        auto turn = [&](int j, uint64_t mate) {
            const uint64_t v = mul_f32x2(rstd2, fma_f32x2(x2[j], wc[j], mul_f32x2(mate, ws[j])));
            y[2 * j] = f32x2_lo(v);
            y[2 * j + 1] = f32x2_hi(v);
        };
        if constexpr (kPairs == kOpposite) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                turn(j, x2[j ^ 4]);
        } else if constexpr (kPairs == kNeighbours) {
            if (p.rot == kHeadDim) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    turn(j, f32x2_pack(x[2 * j + 1], x[2 * j]));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool turned = c0 + 64 * (j >> 2) < p.rot;      // (a piece as a whole)
                    turn(j, turned ? f32x2_pack(x[2 * j + 1], x[2 * j]) : 0);
                }
            }
        } else {
            // (a piece that is not turned: the lane's own, or zeros)
            RawBlock<kBf16> other = kHalves ? cur : RawBlock<kBf16>{};
            constexpr int n = kBf16 ? 1 : 2;     // 16-byte words of a piece
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (k == 1 && p.rot <= 64)
                    break;                       // nothing turns in the second pieces
                const int mate = mate_chunk(k), from = (lane & 24) | (mate & 7);
                const bool turned = c0 + 64 * k < p.rot;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    uint4 a = shuffled(cur.v[i], from);
                    if (p.rot > 64) {
                        const uint4 b = shuffled(cur.v[n + i], from);
                        if (mate >= 8)
                            a = b;
                    }
                    if (kHalves || turned)
                        other.v[n * k + i] = a;
                }
            }
            float z[16];
            unpack<kBf16>(other, z);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                turn(j, f32x2_pack(z[2 * j], z[2 * j + 1]));
        }
        if constexpr (kAppend) {
            if (is_k) {
                // the cache holds what the key would be in the input type: the
                // same bytes as storing it and quantising the stored row.  Even
                // lanes give their second piece for the neighbour's first: block
                // part / 2, or 4 + part / 2 in odd lanes.
                const bool odd = part & 1;
                float v[16];
                if constexpr (kBf16) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j] = bf16x2_bits(y[2 * j], y[2 * j + 1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t got = __shfl_xor_sync(kFullMask, odd ? w[j] : w[4 + j], 1);
                        const uint32_t first = odd ? got : w[j], second = odd ? w[4 + j] : got;
                        v[2 * j] = __uint_as_float(first << 16);
                        v[2 * j + 1] = __uint_as_float(first & 0xffff0000u);
                        v[8 + 2 * j] = __uint_as_float(second << 16);
                        v[8 + 2 * j + 1] = __uint_as_float(second & 0xffff0000u);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float got = __shfl_xor_sync(kFullMask, odd ? y[j] : y[8 + j], 1);
                        v[j] = odd ? got : y[j];
                        v[8 + j] = odd ? y[8 + j] : got;
                    }
                }
                size_t rec;
                int tok;
                const int h = heads - ahead;
                if (live && slot_site(p, p.slot_mapping[t], h, rec, tok, h == 0 && part == 0)) {
                    const uint32_t flip = divide_by_tensor_scale(v, head_tensor_scale(p.hs, false, h, p.gscale));
                    write_nvfp4_block(p.pool + rec, false, tok, (part >> 1) + (odd ? 4 : 0), v, ScaleOfByte(), flip);
                }
                continue;
            }
        }
        if (!live)
            continue;
        if (kBf16 || !is_k)
            store_pieces<true>(out, y);
        else
            store_pieces<false>(out, y);
    }
    }
    }
    if (!ok) {
        // let the copies in flight land before the CTA exits
        if (lane == 0)
            report(p.dev_status, NVFP4KV_DEV_TIMEOUT);
        for (int n = left + end - quad - feed.left; n > 0; --n) {
            mbar_wait_bounded(bar + 8 * st, phase, kWaitLimit);
            if (++st == G::kStages) {
                st = 0;
                phase ^= 1u;
            }
        }
    }
    return ok;
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

// Each warp takes an equal run of the call's quads, token-major, and then of the
// V blocks, one a thread.
template <bool kBf16, bool kAppend, int kPairs>
__global__ void __launch_bounds__(kNrThreads, Ring<kBf16>::kCtas)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p)
{
    extern __shared__ __align__(128) uint8_t nr_ring[];
    __shared__ NrShared sh;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
        for (int k = 0; k < Ring<kBf16>::kStages; ++k)
            mbar_init(smem_addr(&sh.bar[warp][k]), 1);
        fence_mbar_init();
    }
    // (the wait comes before the trigger: a kernel that starts early behind
    // this one finds everything before it complete)
    pdl_wait();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < 2 * kHeadDim; i += kNrThreads) {
        const void *w = i < kHeadDim ? p.q_weight : p.k_weight;
        const int c = i % kHeadDim;
        float v = 1.f;
        if (w != nullptr)
            v = p.weight_bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(w)[c]) << 16)
                              : static_cast<const float *>(w)[c];
        sh.weight[i / kHeadDim][c] = v;
    }
    if (threadIdx.x < kHeadDim / 2)
        sh.freq[threadIdx.x] = p.freq[threadIdx.x];
    __syncthreads();
    const long long quads = static_cast<long long>(p.num_tokens) * p.quads;
    const long long warps = static_cast<long long>(gridDim.x) * kNrWarps, rows = min(warps, quads);
    const long long me = static_cast<long long>(blockIdx.x) * kNrWarps + warp, run = min(me, rows);
    if (!rows_of_warp<kBf16, kAppend, kPairs>(p, sh,
                                              smem_addr(nr_ring) + warp * Ring<kBf16>::kStages * Ring<kBf16>::kStage,
                                              quads * run / rows, quads * min(run + 1, rows) / rows))
        return;
    if constexpr (kAppend) {
        // (warps without rows come first)
        for (long long job = me >= rows ? me - rows : me + warps - rows; job < p.v_jobs; job += warps) {
            const long long item = job * 32 + (threadIdx.x & 31);
            const long long unit = item >> 3;    // pair * hkv + h
            const long long pr = unit / p.hkv;
            if (2 * pr <= p.num_tokens)          // (the early start adds half a pair)
                v_pair_job<kBf16>(p, static_cast<int>(pr), static_cast<int>(unit - pr * p.hkv),
                                  static_cast<int>(item & 7));
        }
    }
}

template <bool kBf16, bool kAppend, int kPairs>
cudaError_t launch_rows(const NormRopeParams &p, long long jobs, int sms, cudaStream_t s)
{
    using G = Ring<kBf16>;
    const auto kernel = norm_rope_kernel<kBf16, kAppend, kPairs>;
    if (G::kSmem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
        if (e != cudaSuccess)
            return e;
    }
    const long long want = (jobs + kNrWarps - 1) / kNrWarps, most = static_cast<long long>(sms) * G::kCtas;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kNrThreads), G::kSmem, s, p);
}

} // namespace

cudaError_t launch_norm_rope(const NormRopeParams &in, cudaStream_t s)
{
    NormRopeParams p = in;
    const int sms = sm_count() > 0 ? sm_count() : 1;
    p.q_quads = (p.hq + 3) / 4;
    p.quads = p.q_quads + (p.hkv + 3) / 4;
    const bool append = p.pool != nullptr;
    p.v_jobs = append ? ((static_cast<long long>(p.num_tokens) + 2) / 2 * p.hkv * 8 + 31) / 32 : 0;
    const long long jobs = static_cast<long long>(p.num_tokens) * p.quads + p.v_jobs;
    auto launch = [&](auto bf16, auto app) {
        if (p.interleaved || p.rot == 0)
            return launch_rows<bf16.value, app.value, kNeighbours>(p, jobs, sms, s);
        return p.rot == kHeadDim ? launch_rows<bf16.value, app.value, kOpposite>(p, jobs, sms, s)
                                 : launch_rows<bf16.value, app.value, kTwoLanes>(p, jobs, sms, s);
    };
    if (append)
        return p.in_bf16 ? launch(std::true_type(), std::true_type()) : launch(std::false_type(), std::true_type());
    return p.in_bf16 ? launch(std::true_type(), std::false_type()) : launch(std::false_type(), std::false_type());
}

} // namespace nvfp4kv
