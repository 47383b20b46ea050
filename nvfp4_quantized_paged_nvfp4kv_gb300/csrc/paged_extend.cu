// Attention of a ragged chunk of tokens over the paged NVFP4 cache itself, on
// the fifth-generation tensor cores (tcgen05).
//
// Sequence b has seq_lens[b] = L cached tokens, the last C = q_indptr[b + 1] -
// q_indptr[b] of them being the chunk; chunk token t sits at position
// n = L - C + t and sees the keys max(0, n - window + 1) .. n (all up to n
// without a window):
//   o = sum_j softmax_j(sm_scale q . k_j) v_j,  k, v = G * E4M3 scale * E2M1 code.
//
// A row is a (chunk token, query head of the kv head's group) pair, taken
// token-major.  A CTA owns rows of one sequence and kv head and a run of 128-key
// tiles, and has two MMA blocks of 128 rows at work: two row blocks that share
// every tile (kKeySplit false), or, where a sequence has no more than 128 rows
// a kv head, the same row block twice, one copy on the even tiles and one on
// the odd ones, joined in shared memory at the end (kKeySplit true).  The tensor
// core works for one block while the other is in its softmax.  Per tile:
//   load      one warp copies the page records (2,304 bytes each, one bulk copy
//             a page) into a ring of 64-key granules, page ids looked up a
//             window of 32 pages ahead
//   convert   four warps expand the codes to f16 in the operands' 128-byte
//             swizzle: K as [128 keys][128 channels], V transposed as
//             [128 channels][128 keys], so that the two tokens that a V byte
//             holds are neighbours in the operand
//   S = Q K^T tcgen05.mma M128 N128 K16 x 8, Q in shared memory
//   softmax   one thread a row, 64 keys at a time: exp2 against a reference
//             0 to 8 log2 units under the largest score of the first keys seen,
//             raised only when the sum of 64 weights passes 2^15 (so that no maximum is
//             taken as a rule), P (f16) back into the columns of S
//   O += P V  tcgen05.mma M128 N128 K16 x 8, P and O in tensor memory
// Tiles of 64 keys with Q in tensor memory, which spare the Q reads, ran at half
// the rate: an M128 N64 MMA takes the tensor core the 64 cycles of an N128 one.
//
// Roundings.  Codes and scales: an E2M1 code (two significant bits) times an
// E4M3 scale (four) is exact in f16.  The scale byte's seven bits moved to
// f16's exponent and mantissa are the scale times 2^-8 without a conversion, so
// K and V are held as value / (256 G) and the factors go to the scores and the
// output in fp32.  Any byte gives a finite value this way (0x7F reads as 480
// where E4M3 has NaN), so what masked places, unwritten slots and pages that
// are not loaded hold cannot reach a row that does not see them.  Q: each row
// times a power of two that puts its largest element in [2^14, 2^15), which
// makes bf16 -> f16 exact but for elements under 2^-28 of the row's largest.
// P is rounded to f16, the type of V beside it (bf16 would hold V too, with P three
// bits coarser); at most 2^15, its largest at least 1: relative 2^-11 down to 2^-14,
// and below by up to 2^-25, which the reference keeps at 2^-10 of the sum of weights
// over all keys (reference_lift).  Scores, sums and O are fp32.
//
// Work split.  A unit is a row tile of one sequence and kv head with all its key
// tiles.  The units' tiles, heads outermost, form one sequence, a unit counting
// four more for its own cost (with one a prompt of 4,096 tokens took 176 us, not
// 154), which is cut into equal runs, one a resident CTA: no wave is left half
// empty and few rows with many keys still occupy every SM (whole units, cut by a
// fixed number where there were few: 2,048 tokens at 32K 1.37 ms, 1.14 in runs).
// A CTA's run begins and ends inside a unit as a rule: of those it leaves O,
// reference and sum in the workspace (at most two pieces), which a second kernel
// joins; the units inside are written directly.  Loads and conversions for the
// next unit run behind the end of the last.  (Its Q by the converter warps, or by
// the softmax warps ahead of the last unit's output, also overlaps, but the state
// it keeps in registers cost every tile 3 to 4%.)
//
// Bound.  2,048 tokens of 48 + 8 heads at 32K: 1,400 TFLOP/s, 73% of a library
// GEMM's rate; a tile's softmax, P V and Q K^T follow one another, and two blocks
// fill most of each other's gaps.  16 tokens each of 12 sequences at 8K: 73 us,
// the conversion of a tile for one block's rows only.
#include "tcgen05.cuh"

namespace nvfp4kv {
namespace {

constexpr int kRowsBlock = 128;                // M of one MMA
constexpr int kKeys = 128;                     // keys of a tile
constexpr int kGranKeys = 64;                  // keys of a granule: what is loaded and converted at a time
constexpr int kGrans = kKeys / kGranKeys;
constexpr int kGranPages = kGranKeys / kPageSize;
constexpr int kConvThreads = 128;
constexpr float kMaxSum = 32768.f;             // of 64 weights, before the reference of the softmax moves
// From here on a reference's last place is two log2 units and more, and what the
// fused s inv - m leaves of the rounding of m would be a weight of its own (past
// f16 from 2^28 on): rows that have such a reference take scores rounded to fp32
// first, of which m is one.
constexpr float kFar = 16777216.f;

constexpr uint32_t kOpBytes = kKeys * kHeadDim * 2;            // 32 KB: a Q, K or V operand tile
constexpr uint32_t kHalfBytes = kOpBytes / 2;                  // its 64-channel (V: 64-key) half: 128 rows of 128 bytes
constexpr uint32_t kRawBytes = kGranPages * kNvfp4Record;      // 9,216
// tensor-memory columns of a block: O (fp32), S (fp32; P overwrites its first 64)
constexpr uint32_t kTmO = 0, kTmS = 128, kTmBlock = 256;

constexpr int kSoftmaxThreads = 2 * kRowsBlock;
constexpr int kConvWarp = kSoftmaxThreads / 32;
constexpr int kStages = 2;                     // converted tiles

template <bool kKeySplit>
struct Shape {
    static constexpr int kRows = kKeySplit ? kRowsBlock : 2 * kRowsBlock;    // of a CTA
    static constexpr int kRaw = kKeySplit ? 6 : 3;                           // loaded granules
    static constexpr int kConvGroups = kKeySplit ? 2 : 1;                    // of 128 threads; two: one a block
    static constexpr int kMmaWarp = kConvWarp + kConvGroups * kConvThreads / 32;
    static constexpr int kLoadWarp = kMmaWarp + 2;                           // one MMA warp a block
    static constexpr int kThreads = 32 * (kLoadWarp + 1);
    static constexpr uint32_t kOffQ = 0;
    static constexpr uint32_t kOffK = kOffQ + kRows / kRowsBlock * kOpBytes;
    static constexpr uint32_t kOffV = kOffK + kStages * kOpBytes;
    static constexpr uint32_t kOffRaw = kOffV + kStages * kOpBytes;
    static constexpr uint32_t kOffBar = kOffRaw + kRaw * kRawBytes;
    enum : int {
        kRawFull = 0, kRawEmpty = kRawFull + kRaw, kKFull = kRawEmpty + kRaw, kVFull = kKFull + kStages,
        kTurn = kVFull + kStages, kQFull = kTurn + kStages, kSFull = kQFull + 2, kPFull = kSFull + 2,
        kHalf = kPFull + 4, kDone = kHalf + 2, kGo = kDone + 2, kExit = kGo + 2, kJoin = kExit + 2, kFree = kJoin + 1,
        kVDone = kFree + 1, kNumBars = kVDone + 2
    };
    static constexpr uint32_t kOffSlot = kOffBar + 8 * kNumBars;             // tensor-memory address, failure flag
    static constexpr uint32_t kOffRun = (kOffSlot + 8 + 15) / 16 * 16;
    // key split: (reference, sum) of both blocks' rows, and the rows' score factors
    static constexpr uint32_t kOffMl = kOffRun + 80, kOffInv = kOffMl + (kKeySplit ? 2 * 8 * kRowsBlock : 0);
    static constexpr uint32_t kSmem = kOffInv + (kKeySplit ? 4 * kRowsBlock : 0) + 1024;   // + slack to align the base
    // (one CTA an SM: all of tensor memory is its own)
    static_assert(kSmem <= 227 * 1024 && 2 * kSmem > 228 * 1024, "shared memory");
};
// the sequences' weights, summed up, and chunks take the operand stages' place while a CTA looks for its run
constexpr uint32_t kTableBytes = (kMaxBatch + 2) * 8;

__device__ __forceinline__ void st_shared128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 32 bytes to global memory, at 32 (wide) or 16.
__device__ __forceinline__ void store_sector(uint8_t *dst, bool wide, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                             uint32_t e, uint32_t f, uint32_t g, uint32_t h)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a), "r"(b), "r"(c),
                     "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(a, b, c, d);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(e, f, g, h);
    }
}

// Bounded wait for a phase.  Another role's failure is looked at only while the
// phase is not there yet: a load of the flag in front of every wait cost a
// quarter of the pipeline's turn-around.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *fail, int32_t *dev_status,
                                         uint32_t limit)
{
    for (uint32_t i = 0; i < limit; ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (*fail)
            return false;
    }
    *fail = 1;
    report(dev_status, NVFP4KV_DEV_TIMEOUT);
    return false;
}

// The same for three phases at once: one after the other each read of a barrier
// would cost its whole latency.
__device__ __forceinline__ bool wait_bars(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb, uint32_t c, uint32_t pc,
                                          volatile int *fail, int32_t *dev_status, uint32_t limit)
{
    for (uint64_t i = 0; i < 64ull * limit; ++i) {       // (test_wait does not wait: more polls to the limit)
        const bool ra = mbar_test_wait(a, pa), rb = mbar_test_wait(b, pb), rc = mbar_test_wait(c, pc);
        if (ra && rb && rc)
            return true;
        if ((i & 63) == 63 && *fail)
            return false;
    }
    *fail = 1;
    report(dev_status, NVFP4KV_DEV_TIMEOUT);
    return false;
}

// One arrival for the warp, after what all its lanes did before.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane)
{
    __syncwarp();
    if (lane == 0)
        mbar_arrive(bar);
}

// A sequence's chunk; false (nothing of it is written) when its index range,
// or its length, is outside what the call was given.
struct Chunk {
    int c0, count, len;
};

__device__ __forceinline__ bool read_chunk(const PagedExtendParams &p, int b, Chunk &c)
{
    c.c0 = p.q_indptr[b];
    const int c1 = p.q_indptr[b + 1];
    c.len = p.seq_lens[b];
    c.count = c1 - c.c0;
    return c.c0 >= 0 && c1 >= c.c0 && c1 <= p.q_rows && c.count <= p.max_q_len && c.len >= 0 &&
           c.len <= p.max_pages * kPageSize;
}

// K of a staged granule, thread pt of 128: two quarter rows of 32 channels.
// Loads and conversions are apart so that all loads of a tile are out before the
// first conversion (one warp a scheduler has no other to hide them behind).
struct RawK {
    uint4 d[2];
    uint32_t s[2];
};

__device__ __forceinline__ void load_k(uint32_t raw, int pt, RawK &k)
{
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint32_t idx = pt + kConvThreads * u, key = idx >> 2, quarter = idx & 3u;
        const uint32_t rec = raw + (key >> 4) * kNvfp4Record;
        k.d[u] = lds128(rec + (key & 15u) * 64u + quarter * 16u);
        k.s[u] = lds_u16(rec + 2048u + (key & 15u) * 8u + 2u * quarter);
    }
}

// ... to f16 [key][channel] at dst (the granule's first key's row).  Lanes of
// the upper channel half of a quarter pair store their chunks in another order,
// so eight lanes meet eight bank groups.
__device__ __forceinline__ void convert_k(const RawK &k, uint32_t dst, int pt)
{
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint32_t idx = pt + kConvThreads * u, key = idx >> 2, quarter = idx & 3u;
        const uint4 d = k.d[u];
        const uint32_t two = k.s[u] & 0x7f7fu;
        const bool swap = quarter & 2u;
        const uint32_t w[4] = {swap ? d.z : d.x, swap ? d.w : d.y, swap ? d.x : d.z, swap ? d.y : d.w};
        const uint32_t lo = two & 0xffu, hi = two >> 8;
        const uint32_t sc[2] = {(swap ? hi : lo) * 0x00800080u, (swap ? lo : hi) * 0x00800080u};
        const uint32_t row = dst + (quarter >> 1) * kHalfBytes + key * 128u;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            uint32_t r0, r1, r2, r3;
            e2m1x8_to_f16x2x4(w[i], r0, r1, r2, r3);
            const uint32_t s = sc[i >> 1];
            const uint32_t chunk = (4u * (quarter & 1u) + (i ^ (quarter & 2u))) ^ (key & 7u);
            st_shared128(row + (chunk << 4), hmul2(r0, s), hmul2(r1, s), hmul2(r2, s), hmul2(r3, s));
        }
    }
}

// V of a staged granule: thread pt takes eight keys (half a page, four token
// pairs), group g of the pairs' rows and half its blocks.
struct RawV {
    uint2 d[4], s[4];
};

__device__ __forceinline__ void load_v(uint32_t raw, int pt, RawV &v)
{
    const uint32_t g = pt & 7, jh = (pt >> 3) & 1, eight = pt >> 4;
    const uint32_t rec = raw + (eight >> 1) * kNvfp4Record, p0 = (eight & 1u) * 4u;
#pragma unroll
    for (uint32_t r = 0; r < 4; ++r) {
        const uint32_t p = p0 + r;
        v.d[r] = lds64(rec + 1024u + p * 128u + ((g + 2u * p) & 7u) * 16u + 8u * jh);
        v.s[r] = lds64(rec + 2176u + p * 16u + 8u * jh);
    }
}

// ... to f16 [channel][key] (a 64-key half of the operand).
__device__ __forceinline__ void convert_v(const RawV &v, uint32_t dst, int pt)
{
    const uint32_t g = pt & 7, jh = (pt >> 3) & 1, eight = pt >> 4;
#pragma unroll
    for (uint32_t half = 0; half < 2; ++half) {
        uint32_t f[4][4];                        // [pair row][(block, w)]: tokens 2p, 2p + 1
#pragma unroll
        for (uint32_t r = 0; r < 4; ++r) {
            const uint32_t sw = (half ? v.s[r].y : v.s[r].x) & 0x7f7f7f7fu;
            const uint32_t s0 = __byte_perm(sw, 0, 0x4140) << 7, s1 = __byte_perm(sw, 0, 0x4342) << 7;
            e2m1x8_to_f16x2x4(half ? v.d[r].y : v.d[r].x, f[r][0], f[r][1], f[r][2], f[r][3]);
            f[r][0] = hmul2(f[r][0], s0);
            f[r][1] = hmul2(f[r][1], s0);
            f[r][2] = hmul2(f[r][2], s1);
            f[r][3] = hmul2(f[r][3], s1);
        }
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            const uint32_t channel = 16u * (4u * jh + 2u * half + (k >> 1)) + 8u * (k & 1u) + g;
            st_shared128(dst + channel * 128u + ((eight ^ g) << 4), f[0][k], f[1][k], f[2][k], f[3][k]);
        }
    }
}

// 64 scores of a row (tensor-memory columns at taddr).
__device__ __forceinline__ void load_scores(uint32_t taddr, float (&s)[64])
{
    uint32_t s0[32], s1[32];
    tmem_ld32(taddr, s0);
    tmem_ld32(taddr + 32, s1);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        s[j] = __uint_as_float(s0[j]);
        s[j + 32] = __uint_as_float(s1[j]);
    }
}

// 2^(s inv - m) of scores, as f16 pairs; their sum (of the unrounded values) is
// returned.  kCare: m may be far from 0.
template <bool kCare, int kN>
__device__ __forceinline__ float weights_of(const float (&s)[kN], float inv, float m, uint32_t (&pw)[kN / 2])
{
    const float mbase = m == -INFINITY ? 0.f : m;
    const bool far = kCare && fabsf(mbase) >= kFar;
    const float pre = far ? inv : 1.f, by = far ? 1.f : inv;     // (a branch for far rows spilled, a product does not)
    const uint64_t pre2 = f32x2_pack(pre, pre), by2 = f32x2_pack(by, by), neg2 = f32x2_pack(-mbase, -mbase);
    uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kN / 2; ++j) {
        uint64_t x = f32x2_pack(s[2 * j], s[2 * j + 1]);
        if (kCare)
            x = mul_f32x2(x, pre2);
        const uint64_t d = fma_f32x2(x, by2, neg2);
        const float a = fast_exp2(f32x2_lo(d)), b = fast_exp2(f32x2_hi(d));
        acc[j & 3] = add_f32x2(acc[j & 3], f32x2_pack(a, b));
        pw[j] = pack_f16x2(a, b);
    }
    const uint64_t a = add_f32x2(add_f32x2(acc[0], acc[1]), add_f32x2(acc[2], acc[3]));
    return f32x2_lo(a) + f32x2_hi(a);
}

// How far under the largest score a new reference is, in log2 units, for a piece of
// so many tiles.  A weight is off by up to 2^-25 as an f16 number, and gone below
// that: over 2^15 keys as much as 2^-10 of the sum of weights, over 2^20 3%.  One
// unit a doubling keeps it at 2^-10, up to 2^23 keys (at nine 64 equal weights would
// be at kMaxSum).  Fewer units leave more room before the reference moves: with eight
// for every piece a 4,096-token prompt of scores 6 log2 units apart took 307 us, not
// 165, with one for 2,048 tokens at 32K 1.31 ms, not 1.23.
__device__ __forceinline__ float reference_lift(int tiles)
{
    constexpr int kFree = (1 << 15) / kKeys;
    return tiles <= kFree ? 0.f : static_cast<float>(min(8, 32 - __clz((tiles - 1) / kFree)));
}

// What a row's softmax keeps: the reference and the sum of weights relative to it.
struct RowSum {
    float m, l;
};

// Bits lo .. hi - 1 (any integers) of 32.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi)
{
    const uint32_t below_hi = hi >= 32 ? ~0u : (hi <= 0 ? 0u : (1u << hi) - 1u);
    const uint32_t below_lo = lo >= 32 ? ~0u : (lo <= 0 ? 0u : (1u << lo) - 1u);
    return below_hi & ~below_lo;
}

// The weights of 64 scores the long way: masked to the keys lo .. hi - 1 of them,
// with references far from 0, and, where a row has no reference yet or its weights
// sum to more than kMaxSum, with the reference raised to `lift` under the
// largest score; O (where has_o), once landed() says that the products so far are in it,
// and l, which are relative to the old one, follow.  A warp together; false when
// landed() gave up.  kKeep: the scores stay in registers between the maximum and
// the weights (row blocks: 0.5% faster; with split keys and their 96 registers they
// spill, 9% slower).
template <bool kKeep, class Landed>
__device__ __forceinline__ bool weights_with_care(uint32_t scores, uint32_t weights, uint32_t o_cols, bool has_o,
                                                  int lo, int hi, float inv, int tiles, RowSum &row, Landed landed)
{
    const uint32_t seen[2] = {bit_range(lo, hi), bit_range(lo - 32, hi - 32)};
    auto load = [&](float (&s)[64]) {
        load_scores(scores, s);
#pragma unroll
        for (int j = 0; j < 64; ++j)
            s[j] = (seen[j >> 5] >> (j & 31)) & 1u ? s[j] : -INFINITY;
    };
    bool raise = row.m == -INFINITY;
    for (bool again = false;; again = true) {
        float s[64];
        if (kKeep)
            load(s);
        if (__any_sync(kFullMask, raise)) {
            if (!kKeep)
                load(s);
            float pm[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                pm[k] = fmax3(fmax3(s[8 * k], s[8 * k + 1], s[8 * k + 2]),
                              fmax3(s[8 * k + 3], s[8 * k + 4], s[8 * k + 5]), fmaxf(s[8 * k + 6], s[8 * k + 7]));
            const float top = __fmul_rn(
                fmax3(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])), inv);
            // (keys, but every score -inf: an infinite query, say; no weights, but not
            // a row that sees nothing)
            if (raise && top == -INFINITY && (seen[0] | seen[1]))
                row.l = NAN;
            raise = raise && top > -INFINITY;
            const float m_new = raise ? (fabsf(top) < kFar ? top - reference_lift(tiles) : top) : row.m;
            const float alpha = raise ? fast_exp2(row.m - m_new) : 1.f;
            row.m = m_new;
            row.l *= alpha;
            if (has_o && __any_sync(kFullMask, raise)) {
                if (!landed())
                    return false;
                tc_fence_after_sync();
#pragma unroll 1
                for (int cb = 0; cb < 4; ++cb) {
                    uint32_t o[32];
                    tmem_ld32(o_cols + 32 * cb, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tmem_st32(o_cols + 32 * cb, o);
                }
                if (kKeep)
                    load(s);                     // (not kept beside O)
            }
        }
        if (!kKeep)
            load(s);
        uint32_t pw[32];
        const float sum = weights_of<true>(s, inv, row.m, pw);
        raise = sum > kMaxSum;
        if (again || !__any_sync(kFullMask, raise)) {
            row.l += sum;
            tmem_st32(weights, pw);              // (over scores that have been read)
            return true;
        }
    }
}

// A row tile of one sequence and kv head, and the piece of its key tiles that
// falls into a CTA's run.
struct Unit {
    int b, h, tile;
    int row0, rows;                      // first row, and rows of the sequence and kv head
    int c0, first_pos;                   // row and position of chunk token 0 (negative position: the chunk is longer)
    int key_begin, key_end;              // keys that some row sees
    int tile_lo, all;                    // first key tile, and how many
    int from, n_tiles;                   // the piece: tiles from .. from + n_tiles - 1 of them

    __device__ __forceinline__ bool whole() const { return n_tiles == all; }

    // Row tile `at` of a sequence with rows.
    template <int kRows>
    __device__ __forceinline__ void set(const PagedExtendParams &p, const Chunk &c, int at)
    {
        tile = at;
        rows = c.count * p.group;
        row0 = at * kRows;
        c0 = c.c0;
        first_pos = c.len - c.count;
        const int t_last = (min(row0 + kRows, rows) - 1) / p.group;
        key_end = max(0, first_pos + t_last + 1);
        key_begin = p.window > 0 ? max(0, first_pos + row0 / p.group - p.window + 1) : 0;
        tile_lo = key_begin / kKeys;
        all = key_end > key_begin ? (key_end + kKeys - 1) / kKeys - tile_lo : 0;
    }
};

// Row tiles of a sequence; 0 for one out of bounds.
template <int kRows>
__device__ __forceinline__ int row_tiles_of(const PagedExtendParams &p, int b, Chunk &c)
{
    return read_chunk(p, b, c) ? (c.count * p.group + kRows - 1) / kRows : 0;
}

// Where a CTA's run begins (c, n: that sequence's chunk and row tiles), and how
// much it holds (in tiles and units).
struct Run {
    int h, b, tile, off;
    long long left;
    Chunk c;
    int n;
};

constexpr int kMinRun = 3;               // a run is at least this long, else fewer CTAs take part
// What a unit costs beside its tiles, in tiles (Q in, O out, the pipeline filled
// anew: some 8 us), and so also what a cut inside a unit costs.
constexpr int kUnitCost = 4;
// A cut moves to its unit's nearer border where it would leave no more than
// kSnap tiles of the unit on one side, or where the unit has no more than kWhole
// (a call without cuts needs no join: 700 tokens of 32 + 8 heads 23 us, 28 with).
constexpr int kSnap = 2, kWhole = 8;

// A place in the sequence of units: `off` into row tile `tile` of sequence b, kv
// head h; `at` counts from the beginning.
struct Place {
    int h, b, tile, off;
    long long at;
    Chunk c;
    int n;                               // row tiles of the sequence
};

// Chunks that find_run keeps in shared memory for find_cut: with nearly all of it
// taken there is no first-level cache, and a second read costs as much as the
// first.
constexpr int kKeptChunks = 1024;

// Where the cut at `at` of `head` x hkv places falls (whole warp); table: batch +
// 1 running sums; kept: the first kKeptChunks sequences' chunks.
template <int kRows>
__device__ __forceinline__ Place find_cut(const PagedExtendParams &p, long long at, long long head,
                                          const long long *table, const Chunk *kept, int lane)
{
    Place r{p.hkv, 0, 0, 0, at, {0, 0, 0}, -1};
    if (at >= head * p.hkv)
        return r;
    r.h = static_cast<int>(at / head);
    long long rest = at - r.h * head;
    int x = 0, y = p.batch;              // the last sequence that begins at or before `rest`
    while (y - x > 1) {
        const int mid = (x + y) >> 1;
        if (table[mid] <= rest)
            x = mid;
        else
            y = mid;
    }
    r.b = x;
    rest -= table[x];
    Chunk c = kept[min(x, kKeptChunks - 1)];
    const int n = x < kKeptChunks ? (c.count * p.group + kRows - 1) / kRows : row_tiles_of<kRows>(p, x, c);
    r.c = c;
    r.n = n;
    for (int i0 = 0; i0 < n; i0 += 32) {
        Unit u{};
        int w = 0;
        if (i0 + lane < n) {
            u.set<kRows>(p, c, i0 + lane);
            w = u.all + kUnitCost;
        }
        long long incl = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(kFullMask, incl, o);
            if (lane >= o)
                incl += v;
        }
        const unsigned past = __ballot_sync(kFullMask, i0 + lane < n && incl > rest);
        if (past) {
            const int hit = __ffs(past) - 1, size = __shfl_sync(kFullMask, w, hit);
            r.tile = i0 + hit;
            r.off = static_cast<int>(rest - __shfl_sync(kFullMask, incl - w, hit));
            const int before = r.off - kUnitCost, behind = size - r.off;     // tiles
            if (before <= kSnap || behind <= kSnap || before + behind <= kWhole) {
                const bool down = before <= behind;
                r.at += down ? -r.off : behind;
                r.tile += !down;                 // (up: the next one's beginning)
                r.off = 0;
            }
            break;
        }
        rest -= __shfl_sync(kFullMask, incl, 31);
    }
    return r;
}

// Finds the run of worker `worker` of `workers`; whole CTA.  In shared memory:
// `table`, batch + 1 sums, and `kept`, kKeptChunks chunks.
template <int kRows>
__device__ __forceinline__ void find_run(const PagedExtendParams &p, int worker, int workers, long long *table,
                                         Chunk *kept, Run *run)
{
    __shared__ long long part[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    // weights: a group of lanes a sequence, the more lanes the fewer sequences
    int width = 32;
    while (width > 1 && blockDim.x / width < p.batch)
        width >>= 1;
    const int sub = lane & (width - 1), groups = blockDim.x / width;
    for (int b0 = 0; b0 < p.batch; b0 += groups) {
        const int b = b0 + static_cast<int>(threadIdx.x) / width;
        long long w = 0;
        if (b < p.batch) {
            Chunk c;
            const int n = row_tiles_of<kRows>(p, b, c);
            if (n == 0 && sub == 0 && worker == 0 && !read_chunk(p, b, c))
                report(p.dev_status, NVFP4KV_DEV_BAD_LEN);
            if (sub == 0 && b < kKeptChunks)
                kept[b] = {c.c0, n > 0 ? c.count : 0, c.len};
            Unit u{};
            for (int i = sub; i < n; i += width) {
                u.set<kRows>(p, c, i);
                w += u.all + kUnitCost;
            }
        }
        for (int o = 1; o < width; o <<= 1)
            w += __shfl_xor_sync(kFullMask, w, o);
        if (b < p.batch && sub == 0)
            table[b + 1] = w;
    }
    if (threadIdx.x == 0)
        table[0] = 0;
    __syncthreads();
    // their running sum
    long long carry = 0;
    for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        long long x = b < p.batch ? table[b + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(kFullMask, x, o);
            if (lane >= o)
                x += y;
        }
        if (lane == 31)
            part[warp] = x;
        __syncthreads();
        long long total = 0, before = carry;
        for (int k = 0; k < warps; ++k) {
            before += k < warp ? part[k] : 0;
            total += part[k];
        }
        if (b < p.batch)
            table[b + 1] = before + x;
        carry += total;
        __syncthreads();
    }
    // the run's two ends, by a warp each
    if (warp < 2) {
        const long long head = table[p.batch], all = head * p.hkv;
        const long long use = min(static_cast<long long>(workers), max(1LL, all / kMinRun));
        const Place r = find_cut<kRows>(p, all * min(worker + warp, static_cast<int>(use)) / use, head, table, kept,
                                        lane);
        if (lane == 0) {
            if (warp == 0) {
                run->h = r.h;
                run->b = r.b;
                run->tile = r.tile;
                run->off = r.off;
                run->c = r.c;
                run->n = r.n;
            }
            part[warp] = r.at;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0)
        run->left = part[1] - part[0];
    __syncthreads();
}

// A softmax thread's row.
struct Row {
    bool live;
    int t;                               // chunk token
    int64_t at;                          // row of q and out, in heads
};

template <int kRows>
__device__ __forceinline__ Row row_of(const PagedExtendParams &p, const Unit &u, int tid)
{
    const int r = u.row0 + tid % kRows, in = min(r, u.rows - 1);
    Row w;
    w.live = r < u.rows;
    w.t = in / p.group;
    w.at = static_cast<int64_t>(u.c0 + w.t) * p.hq + u.h * p.group + (in - w.t * p.group);
    return w;
}

// A CTA's way through its run.
struct Walk {
    Unit u;
    Chunk c;
    int n, at, off;                      // row tiles of the sequence, the next one, and its place to begin at
    long long left;

    __device__ __forceinline__ explicit Walk(const Run &r) : u{}, c(r.c), n(r.n), at(r.tile), off(r.off), left(r.left)
    {
        u.h = r.h;
        u.b = r.b;
    }
};

// The next unit with keys (its piece in w.u), or false at the end of the run.
// Rows that see no key are written on the way, by threads 0 .. kRows - 1.  (One
// copy for all roles.)
template <int kRows>
__device__ __forceinline__ bool next_unit(const PagedExtendParams &p, Walk &w, int tid)
{
    Unit &u = w.u;
    while (w.left > 0 && u.h < p.hkv) {
        if (w.n < 0)
            w.n = row_tiles_of<kRows>(p, u.b, w.c);
        if (w.at >= w.n) {
            w.n = -1;
            w.at = w.off = 0;
            if (++u.b == p.batch) {
                u.b = 0;
                ++u.h;
            }
            continue;
        }
        u.set<kRows>(p, w.c, w.at);
        // the first places of a unit are its own cost, then come its tiles
        const int take = static_cast<int>(min(w.left, static_cast<long long>(u.all + kUnitCost - w.off)));
        u.from = max(0, w.off - kUnitCost);
        u.n_tiles = max(0, w.off + take - kUnitCost) - u.from;
        w.left -= take;
        ++w.at;
        w.off = 0;
        if (u.all == 0 && tid < kRows) {
            const Row row = row_of<kRows>(p, u, tid);
            const int words = p.out_f32 ? kHeadDim / 4 : kHeadDim / 8;
            uint4 *d =
                reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + row.at * kHeadDim * (p.out_f32 ? 4 : 2));
            for (int k = 0; row.live && k < words; ++k)
                d[k] = make_uint4(0, 0, 0, 0);
        }
        if (u.n_tiles > 0)
            return true;
    }
    return false;
}

// The workspace: for each CTA two pieces of (O [rows][128], then (reference,
// sum) [rows]) -- the one that begins inside its unit and the one that begins
// with it but does not end it -- and then a note of each CTA.
template <int kRows>
constexpr size_t kPieceFloats = static_cast<size_t>(kRows) * (kHeadDim + 2);

struct Note {
    int tail;                            // 1: the second piece is there, of the rows below
    int h, row0, rows, c0;
    int head;                            // 1: the first piece is there, 2: and it ends its unit
    int pad[2];
};

template <int kRows>
__device__ __forceinline__ Note *notes_of(const PagedExtendParams &p)
{
    return reinterpret_cast<Note *>(p.partials + 2 * kPieceFloats<kRows> * p.workers);
}

template <bool kKeySplit>
__global__ void __launch_bounds__(Shape<kKeySplit>::kThreads, 1)
    paged_extend_kernel(const __grid_constant__ PagedExtendParams p)
{
    using S = Shape<kKeySplit>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw_addr);
    volatile int *fail = reinterpret_cast<volatile int *>(gbase + S::kOffSlot + 4);
    auto B = [&](int k) { return base + S::kOffBar + 8 * k; };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kRows = S::kRows;
    Run *run = reinterpret_cast<Run *>(gbase + S::kOffRun);
    if (tid == 0) {
        for (int k = 0; k < S::kRaw; ++k) {
            mbar_init(B(S::kRawFull + k), 1);
            mbar_init(B(S::kRawEmpty + k), kConvThreads / 32);
        }
        for (int k = 0; k < kStages; ++k) {
            mbar_init(B(S::kKFull + k), kConvThreads / 32);
            mbar_init(B(S::kVFull + k), kConvThreads / 32);
            mbar_init(B(S::kTurn + k), kKeySplit ? 1 : 2);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(B(S::kQFull + k), (kKeySplit ? 2 : 1) * kRowsBlock / 32);
            mbar_init(B(S::kSFull + k), 1);
            mbar_init(B(S::kPFull + k), kRowsBlock / 32);
            mbar_init(B(S::kPFull + 2 + k), kRowsBlock / 32);
            mbar_init(B(S::kHalf + k), 1);
            mbar_init(B(S::kDone + k), 1);
            mbar_init(B(S::kGo + k), 1);
            mbar_init(B(S::kExit + k), 1);
            mbar_init(B(S::kVDone + k), 1);
        }
        mbar_init(B(S::kJoin), kSoftmaxThreads / 32);
        mbar_init(B(S::kFree), kSoftmaxThreads / 32);
        *fail = 0;
        fence_mbar_init();
    }
    // nothing before this reads or writes what other kernels do
    pdl_wait();
    if (tid == 0 && p.partials != nullptr) {
        Note *note = notes_of<kRows>(p) + blockIdx.x;
        note->tail = note->head = 0;
    }
    find_run<kRows>(p, blockIdx.x, gridDim.x, reinterpret_cast<long long *>(gbase + S::kOffK),
                    reinterpret_cast<Chunk *>(gbase + S::kOffK + kTableBytes), run);
    static_assert(kTableBytes + kKeptChunks * sizeof(Chunk) <= 2 * kStages * kOpBytes && sizeof(Run) <= 80, "tables");
    const Run start = *run;
    // The units of this CTA's run, one after the other: fn(unit) for each with
    // keys, until it returns false.
    auto for_units = [&](auto fn) {
        Walk w(start);
        while (next_unit<kRows>(p, w, tid)) {
            const Unit u = w.u;                  // (a copy in registers: the walk's own is in memory)
            if (!fn(u))
                return false;
        }
        return true;
    };

    // the rows of Q to come, into L2: the first unit's now, later the next row
    // tile's while the last one is worked on
    auto ask_for_q = [&](const Unit &u) {
        if (tid >= kRows)
            return;
        const Row row = row_of<kRows>(p, u, tid);
        if (row.live) {
            const uint16_t *q = p.q + row.at * kHeadDim;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q + kHeadDim / 2));
        }
    };
    if (start.left > 0 && start.tile < start.n) {
        Unit u{};
        u.h = start.h;
        u.set<kRows>(p, start.c, start.tile);
        ask_for_q(u);
    }
    if (warp == S::kMmaWarp)
        tmem_alloc(base + S::kOffSlot, 2 * kTmBlock);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(gbase + S::kOffSlot);

    if (warp == S::kLoadWarp) {
        // granules in order; lane l looks up page l % 4 of a unit's granule 8 w +
        // l / 4, a window w ahead
        int issued = 0;
        for_units([&](const Unit &u) {
            const int page_lo = u.key_begin / kPageSize, page_hi = (u.key_end + kPageSize - 1) / kPageSize;
            const int n_grans = u.n_tiles * kGrans, first_page = (u.tile_lo + u.from) * (kKeys / kPageSize);
            const int32_t *table = p.block_table + static_cast<size_t>(u.b) * p.max_pages;
            auto lookup = [&](int i) {
                const int pg = first_page + i * kGranPages + (lane & 3);
                return i < n_grans && pg >= page_lo && pg < page_hi ? __ldg(table + pg) : 0;
            };
            int cur = 0, nxt = lookup(lane >> 2);
            for (int i = 0; i < n_grans; ++i, ++issued) {
                if ((i & 7) == 0) {
                    cur = nxt;
                    nxt = lookup(i + 8 + (lane >> 2));
                    if (static_cast<unsigned>(cur) >= static_cast<unsigned>(p.num_pages)) {
                        report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);
                        cur = 0;
                    }
                }
                const int st = issued % S::kRaw;
                // the stage was last read by the converters kRaw granules ago
                bool ok = true;
                if (issued >= S::kRaw)
                    ok = wait_bar(B(S::kRawEmpty + st), (issued / S::kRaw - 1) & 1, fail, p.dev_status, p.wait_limit);
                if (!__all_sync(kFullMask, ok))
                    return false;
                const int pg0 = first_page + i * kGranPages;
                // (0 where no row sees the granule)
                const int n = max(0, min(pg0 + kGranPages, page_hi) - max(pg0, page_lo));
                if (lane == 0)
                    mbar_arrive_expect_tx(B(S::kRawFull + st), n * kNvfp4Record);
                __syncwarp();
                const int pg = pg0 + (lane & 3);
                if ((lane >> 2) == (i & 7) && pg >= page_lo && pg < page_hi)
                    bulk_g2s(base + S::kOffRaw + st * kRawBytes + (lane & 3) * kNvfp4Record,
                             p.pool + (static_cast<size_t>(cur) * p.hkv + u.h) * kNvfp4Record, kNvfp4Record,
                             B(S::kRawFull + st));
            }
            return true;
        });
        // the next kernel's launch overlaps the last tiles (it waits for this
        // one's end before it reads anything)
        pdl_launch_dependents();
        // nothing issued may still be in flight when the CTA exits
        for (int i = max(0, issued - S::kRaw); i < issued; ++i)
            if (!mbar_wait_bounded(B(S::kRawFull + i % S::kRaw), (i / S::kRaw) & 1, kWaitLimit))
                report(p.dev_status, NVFP4KV_DEV_TIMEOUT);
        __syncwarp();
    } else if (warp >= S::kMmaWarp) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_f16(kRowsBlock, 128, false);     // both products: N = 128, K-major
            const int k = warp - S::kMmaWarp;                       // the block
            const uint32_t tb = tmem + k * kTmBlock, qb = base + S::kOffQ + (kKeySplit ? 0 : k) * kOpBytes;
            auto wait = [&](int bar, uint32_t parity) {
                return wait_bar(B(bar), parity, fail, p.dev_status, p.wait_limit);
            };
            // S of tile x; then turn x, which frees K of tile x and V of the
            // block's tile before it.  (One commit for both.)
            auto qk = [&](int x, bool turns) {
                const uint32_t kb = base + S::kOffK + (x & 1) * kOpBytes;
                tc_fence_after_sync();
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    if (s == 4 && turns)
                        mbar_arrive(B(S::kGo + 1 - k));
                    const uint32_t off = (s >> 2) * kHalfBytes + (s & 3) * 32;
                    umma_f16(tb + kTmS, smem_desc(qb + off, 16, 1024), smem_desc(kb + off, 16, 1024), idesc, s > 0);
                }
                umma_commit(B(S::kSFull + k));
                umma_commit(B(S::kTurn + (x & 1)));
            };
            // P V over the keys 64 half .. + 63 of tile x
            auto pv = [&](int x, int half, bool accumulate) {
                const uint32_t vb = base + S::kOffV + (x & 1) * kOpBytes + half * kHalfBytes;
                tc_fence_after_sync();
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    umma_f16_ts(tb + kTmO, tb + kTmS + 32 * half + 8 * s, smem_desc(vb + 32 * s, 16, 1024), idesc,
                                accumulate || s > 0);
            };
            // P V of a tile, then Q K^T of the block's next one, whose S
            // overwrites that P in issue order.  One thread for both blocks
            // left the tensor core idle through the waits (a barrier takes 250
            // cycles to read beside the MMAs' own shared-memory traffic); two
            // threads without a rule fell into step, both blocks in their
            // softmax at once.  So the blocks take turns: a block issues when
            // the other one is half through the Q K^T of its own turn.
            // Batch n of a block (its P V and Q K^T of one tile step) follows batch
            // n - 1 (block 0) or n (block 1) of the other.  With row blocks K of
            // the next tile is there as a rule, and comes after V of this one from
            // the same converter warps: one wait covers both.
            // A tile's number x counts the CTA's tiles (row blocks), or twice the
            // block's own, plus the block (key split): its stage is x mod 2.
            constexpr int step = kKeySplit ? 2 : 1;
            int ib = 0, un = 0, batch = 0;               // the block's tiles, units and batches so far
            const int go_lag = k == 0 ? 1 : 0;
            for_units([&](const Unit &u) {
                const int mine = kKeySplit ? (u.n_tiles + 1 - k) / 2 : u.n_tiles;
                const bool turns = !kKeySplit || u.n_tiles > 1;          // both blocks have tiles
                auto number = [&](int i) { return kKeySplit ? 2 * i + k : i; };
                auto go = [&]() { return !turns || batch < go_lag || wait(S::kGo + k, (batch - go_lag) & 1); };
                // (every phase is waited for, also by a block without tiles)
                if (!wait(S::kQFull + (kKeySplit ? 0 : k), un++ & 1))
                    return false;
                if (mine == 0)
                    return true;
                const int x0 = number(ib);
                if (!wait(S::kKFull + (x0 & 1), (x0 >> 1) & 1) || !go())
                    return false;
                qk(x0, turns);
                batch += turns;
                for (int j = 0; j < mine; ++j, batch += turns) {
                    const int i = ib + j, x = number(i), next = x + step;
                    const bool more = j + 1 < mine;
                    const uint32_t p_bar = B(S::kPFull + k), p_par = i & 1;
                    const bool waits = turns && batch >= go_lag;
                    const uint32_t go_bar = waits ? B(S::kGo + k) : p_bar;
                    const uint32_t go_par = waits ? (batch - go_lag) & 1 : p_par;
                    const bool k_first = !kKeySplit && more;
                    const uint32_t kv_bar = k_first ? B(S::kKFull + (next & 1)) : B(S::kVFull + (x & 1));
                    const uint32_t kv_par = k_first ? (next >> 1) & 1 : (x >> 1) & 1;
                    if (!wait_bars(p_bar, p_par, go_bar, go_par, kv_bar, kv_par, fail, p.dev_status, p.wait_limit))
                        return false;
                    pv(x, 0, j > 0);
                    umma_commit(B(S::kHalf + k));
                    // (with split keys K of the next tile is there by now as a rule)
                    if (!(kKeySplit && more ? wait_bars(B(S::kPFull + 2 + k), i & 1, B(S::kPFull + 2 + k), i & 1,
                                                        B(S::kKFull + (next & 1)), (next >> 1) & 1, fail, p.dev_status,
                                                        p.wait_limit)
                                            : wait(S::kPFull + 2 + k, i & 1)))
                        return false;
                    pv(x, 1, true);
                    if (kKeySplit)
                        umma_commit(B(S::kVDone + k));
                    if (more)
                        qk(next, turns);
                    else if (turns)
                        mbar_arrive(B(S::kGo + 1 - k));
                }
                umma_commit(B(S::kDone + k));
                ib += mine;
                if (kKeySplit && turns && k == 1 && (u.n_tiles & 1)) {
                    // the other block had a tile more: a batch without work keeps the turns even
                    if (!go())
                        return false;
                    mbar_arrive(B(S::kGo + 1 - k));
                    ++batch;
                }
                return true;
            });
            // nothing of this thread's may still run when tensor memory is freed
            umma_commit(B(S::kExit + k));
            if (!mbar_wait_bounded(B(S::kExit + k), 0, kWaitLimit))
                report(p.dev_status, NVFP4KV_DEV_TIMEOUT);
        }
        __syncwarp();
    } else if (warp >= kConvWarp) {
        const int pt = (tid - kSoftmaxThreads) % kConvThreads;
        auto wait_warp = [&](int k, uint32_t parity) {
            return __all_sync(kFullMask, wait_bar(B(k), parity, fail, p.dev_status, p.wait_limit));
        };
        // (the turn of tile x needs tile x's K, so a turn asked for here is at
        // most kStages behind the last one done: its barrier has not come
        // round again)
        auto wait_turn = [&](int x) { return wait_warp(S::kTurn + (x & 1), (x >> 1) & 1); };
        // tiles by their number x (see the MMA warps), granules by the place y of
        // their tile in the CTA's run
        auto stage = [&](int gr) { return base + S::kOffRaw + gr % S::kRaw * kRawBytes; };
        // A tile's bytes go to registers as soon as they are there, so that the
        // ring's stages are free for the copies to come while conversions wait
        // for their operand stages.
        RawK kx[kGrans];
        RawV vx[kGrans];
        auto take_k = [&](int y) {
#pragma unroll
            for (int u = 0; u < kGrans; ++u) {
                const int gr = y * kGrans + u;
                if (!wait_warp(S::kRawFull + gr % S::kRaw, (gr / S::kRaw) & 1))
                    return false;
                load_k(stage(gr), pt, kx[u]);
            }
            return true;
        };
        auto take_v = [&](int y) {
#pragma unroll
            for (int u = 0; u < kGrans; ++u)
                load_v(stage(y * kGrans + u), pt, vx[u]);
            fence_async_shared();                // the reads before the stages' next copies
#pragma unroll
            for (int u = 0; u < kGrans; ++u)
                warp_arrive(B(S::kRawEmpty + (y * kGrans + u) % S::kRaw), lane);
        };
        // K of tile x: its stage was last read in the turn of tile x - 2
        auto make_k = [&](int x) {
            if (x >= kStages && !wait_turn(x - kStages))
                return false;
#pragma unroll
            for (int u = 0; u < kGrans; ++u)
                convert_k(kx[u], base + S::kOffK + (x & 1) * kOpBytes + u * kGranKeys * 128, pt);
            fence_async_shared();
            warp_arrive(B(S::kKFull + (x & 1)), lane);
            return true;
        };
        // V of tile x: its stage was last read by P V of tile x - 2, which turn
        // x - 1 follows; a block with stages of its own has its word for it
        auto make_v = [&](int x) {
            if (x >= kStages && !(kKeySplit ? wait_warp(S::kVDone + (x & 1), ((x >> 1) - 1) & 1) : wait_turn(x - 1)))
                return false;
#pragma unroll
            for (int u = 0; u < kGrans; ++u)
                convert_v(vx[u], base + S::kOffV + (x & 1) * kOpBytes + u * kHalfBytes, pt);
            fence_async_shared();
            warp_arrive(B(S::kVFull + (x & 1)), lane);
            return true;
        };
        int yb = 0, ib = 0;                      // the CTA's tiles, and the group's, so far
        for_units([&](const Unit &u) {
            if constexpr (kKeySplit) {
                // each group makes its block's tiles: V of one as soon as P V of
                // the one before is done, K of the next after Q K^T of this one
                // (one group for both blocks was what they waited for)
                const int k = (tid - kSoftmaxThreads) / kConvThreads, end = yb + u.n_tiles;
                int y = yb + k, x = 2 * ib + k;
                auto next_k = [&]() {
                    if (!take_k(y))
                        return false;
                    take_v(y);
                    return make_k(x);
                };
                bool ok = y >= end || next_k();
                while (ok && y < end) {
                    ok = make_v(x);
                    y += 2;
                    x += 2;
                    ++ib;
                    if (ok && y < end)
                        ok = next_k();
                }
                yb = end;
                return ok;
            } else {
                const int end = yb + u.n_tiles;
                for (; yb < end; ++yb) {
                    if (!take_k(yb))
                        return false;
                    take_v(yb);
                    if (!make_k(yb) || !make_v(yb))
                        return false;
                }
                return true;
            }
        });
    } else {
        const int blk = warp >> 2, r = tid % kRowsBlock;
        const uint32_t tb = tmem + blk * kTmBlock + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        // the warp leaves together: its tensor-memory accesses are warp-wide
        auto wait_warp = [&](int k, uint32_t parity) {
            return __all_sync(kFullMask, wait_bar(B(k), parity, fail, p.dev_status, p.wait_limit));
        };
        int ib = 0, un = 0, dn = 0;              // the block's tiles, units, and units with tiles, so far
        float2 *ml = reinterpret_cast<float2 *>(gbase + S::kOffMl);
        volatile float *invs = reinterpret_cast<volatile float *>(gbase + S::kOffInv);
        for_units([&](const Unit &u) {
        const Row row = row_of<kRows>(p, u, tid);
        const bool has_row = row.live;
        const int64_t out_row = row.at;
        // With split keys both blocks read both blocks' O at the end of a unit, and
        // share Q: the last unit must be over for both.
        if (kKeySplit && un > 0 && !wait_warp(S::kFree, (un - 1) & 1))
            return false;
        // The rows of Q, each scaled by a power of two; inv takes this thread's
        // scores to log2 units.  A warp loads its 32 rows two at a time, half a
        // warp a row (a row a thread, 16 bytes at a time, took 5 us); with split
        // keys the blocks take half of the rows each.
        const unsigned live = __ballot_sync(kFullMask, has_row);
        const uint32_t stage = base + S::kOffQ + (kKeySplit ? 0 : blk) * kOpBytes;
        float inv;
        {
            constexpr int kN = kKeySplit ? 8 : 16;
            const int piece = lane & 15, first = kKeySplit ? 16 * blk : 0;
            uint4 w[kN];
            // (places of the tile's rows from its first token's on pass no 32 bits)
            const int64_t start = static_cast<int64_t>(u.c0 + u.row0 / p.group) * p.hq + u.h * p.group;
            const uint4 *from = reinterpret_cast<const uint4 *>(p.q + start * kHeadDim) + piece;
            const int rel = static_cast<int>(out_row - start);
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int of = first + 2 * i + (lane >> 4);
                const int at = __shfl_sync(kFullMask, rel, of);
                w[i] = make_uint4(0, 0, 0, 0);
                if ((live >> of) & 1u)
                    w[i] = __ldg(from + static_cast<int64_t>(at) * (kHeadDim / 8));
            }
            const float ks = p.hs.per_head ? p.hs.k[u.h] : p.gscale;
            const float to_log2 = 256.f * ks * fabsf(p.qscale);
            // each row's largest |q| (bf16 bits): kN reductions over half a warp at
            // once, halving the rows a lane holds at every exchange; lane l ends
            // with row first + 2 (l mod kN) + l / 16
            uint32_t top[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const uint32_t m2 = __vmaxu2(__vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                                             __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu));
                top[i] = max(m2 & 0xffffu, m2 >> 16);
            }
#pragma unroll
            for (int o = kN / 2; o > 0; o >>= 1) {
                const bool upper = lane & o;
#pragma unroll
                for (int i = 0; i < o; ++i) {
                    const uint32_t got = __shfl_xor_sync(kFullMask, upper ? top[i] : top[i + o], o);
                    top[i] = max(upper ? top[i + o] : top[i], got);
                }
            }
            if (kN == 8)
                top[0] = max(top[0], __shfl_xor_sync(kFullMask, top[0], 8));
            // 2^e puts it into [2^14, 2^15)
            const int e = min(14 - (static_cast<int>(top[0] >> 7) - 127), 112);
            const float unscaled = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * to_log2;
            float sc = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            sc = p.qscale < 0.f ? -sc : sc;      // scores keep their order: references are taken before inv
            if (unscaled == 0.f)
                sc = 0.f;                        // all scores are 0
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const float f = __shfl_sync(kFullMask, sc, (lane & 16) | i);
                auto two = [&](uint32_t q2) {
                    return pack_f16x2(__uint_as_float(q2 << 16) * f, __uint_as_float(q2 & 0xffff0000u) * f);
                };
                const uint32_t at = 32u * (warp & 3) + first + 2u * i + (lane >> 4);
                st_shared128(stage + (piece >> 3) * kHalfBytes + at * 128u + (((piece & 7u) ^ (at & 7u)) << 4),
                             two(w[i].x), two(w[i].y), two(w[i].z), two(w[i].w));
            }
            inv = unscaled == 0.f ? 1.f : unscaled;
            if constexpr (kKeySplit) {
                if (!(lane & 8))                 // (read once the first scores are there)
                    invs[32 * (warp & 3) + first + 2 * (lane & 7) + (lane >> 4)] = inv;
            } else {
                inv = __shfl_sync(kFullMask, inv, ((lane & 1) << 4) | (lane >> 1));
            }
            fence_async_shared();
            warp_arrive(B(S::kQFull + (kKeySplit ? 0 : blk)), lane);
        }
        if (u.row0 + kRows < u.rows) {
            Unit after = u;
            after.row0 += kRows;
            ask_for_q(after);
        }
        const int pos = u.first_pos + row.t;     // keys lo .. pos are visible
        const int lo = p.window > 0 ? pos - p.window + 1 : 0;
        float m_used = -INFINITY, l = 0.f;
        bool ok = true;
        const int my_tiles = kKeySplit ? (u.n_tiles + 1 - blk) / 2 : u.n_tiles;
        for (int j = 0; ok && j < my_tiles; ++j) {
            const int i = ib + j;
            if (!(ok = wait_warp(S::kSFull + blk, i & 1)))
                break;
            tc_fence_after_sync();
            if (kKeySplit && j == 0)
                inv = invs[r];
            const int k0 = (u.tile_lo + u.from + (kKeySplit ? 2 * j + blk : j)) * kKeys;
            const int hi_j = pos + 1 - k0, lo_j = lo - k0;
            // weights of keys 0 .. 63 go over the columns of scores 0 .. 31, of
            // keys 64 .. 127 over those of scores 32 .. 63
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
                const uint32_t at = tb + kTmS + 64 * hf, to = tb + kTmS + 32 * hf;
                const int lo_h = lo_j - 64 * hf, hi_h = hi_j - 64 * hf;
                bool care = !(fabsf(m_used) < kFar) || lo_h > 0 || hi_h < 64;     // (no reference yet: -inf)
                if (!__any_sync(kFullMask, care)) {
                    float s[64];
                    uint32_t pw[32];
                    load_scores(at, s);
                    const float sum = weights_of<false>(s, inv, m_used, pw);
                    care = __any_sync(kFullMask, sum > kMaxSum);
                    if (!care) {
                        l += sum;
                        tmem_st32(to, pw);
                    }
                } else {
                    care = true;
                }
                if (care) {
                    // O is there after the unit's first products: of the last tile
                    // (S of this one was committed after them), and of this tile's
                    // first half, which may still be under way
                    RowSum sum{m_used, l};
                    ok = weights_with_care<!kKeySplit>(at, to, tb + kTmO, j > 0 || hf == 1, lo_h, hi_h, inv, u.n_tiles,
                                                       sum, [&] { return hf == 0 || wait_warp(S::kHalf + blk, i & 1); });
                    if (!ok)
                        break;
                    m_used = sum.m;
                    l = sum.l;
                }
                tmem_wait_st();
                tc_fence_before_sync();
                warp_arrive(B(S::kPFull + 2 * hf + blk), lane);
            }
            if (!ok)
                break;
        }
        // The block's products have landed; with split keys the other block's too,
        // and each block puts half of the channels together.
        if (ok && my_tiles > 0)
            ok = wait_warp(S::kDone + blk, dn++ & 1);
        float w0 = 1.f, w1 = 0.f;                // weights of the blocks' O (row blocks: of its own)
        if constexpr (kKeySplit) {
            if (ok) {
                ml[kRowsBlock * blk + r] = make_float2(m_used, l);
                tc_fence_before_sync();
                warp_arrive(B(S::kJoin), lane);
                ok = wait_warp(S::kJoin, un & 1);
            }
            if (ok) {
                const float2 a = ml[r], b = ml[kRowsBlock + r];
                m_used = fmaxf(a.x, b.x);
                w0 = a.x == -INFINITY ? 0.f : fast_exp2(a.x - m_used);
                w1 = b.x == -INFINITY ? 0.f : fast_exp2(b.x - m_used);
                l = (a.y != a.y || b.y != b.y) ? NAN : a.y * w0 + b.y * w1;
            }
        }
        tc_fence_after_sync();
        if (ok) {
            const float vs = (p.hs.per_head ? p.hs.v[u.h] : p.gscale) * 256.f;
            const bool whole = u.whole();
            const float f = !whole ? vs : (l > 0.f ? vs / l : (l == 0.f ? 0.f : l));   // a NaN sum stays NaN
            const float f0 = w0 * f, f1 = w1 * f;
            const uint32_t to = kKeySplit ? tb - blk * kTmBlock : tb;    // (the first block's)
            const int piece = 2 * blockIdx.x + (u.from > 0 ? 0 : 1), rr = tid % kRows;
            float *part = p.partials + kPieceFloats<kRows> * piece;
            if (has_row && !whole && (!kKeySplit || blk == 0))
                reinterpret_cast<float2 *>(part + kRows * kHeadDim)[rr] = make_float2(m_used, l);
            if (!whole && tid == 0) {
                Note *note = notes_of<kRows>(p) + blockIdx.x;
                if (u.from > 0) {
                    note->head = u.from + u.n_tiles == u.all ? 2 : 1;
                } else {
                    note->h = u.h;
                    note->row0 = u.row0;
                    note->rows = u.rows;
                    note->c0 = u.c0;
                    note->tail = 1;
                }
            }
            // A row a thread, 32 bytes (a whole sector) a store.
            const bool f32 = !whole || p.out_f32, wide = !whole || (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
            uint8_t *dst = whole ? static_cast<uint8_t *>(p.out) + out_row * kHeadDim * (p.out_f32 ? 4 : 2)
                                 : reinterpret_cast<uint8_t *>(part + rr * kHeadDim);
#pragma unroll 1
            for (int cb = kKeySplit ? 2 * blk : 0; cb < (kKeySplit ? 2 * blk + 2 : 4); ++cb) {
                uint32_t o[32];
                __syncwarp();                    // (lanes without a row skip the stores)
                tmem_ld32(to + kTmO + 32 * cb, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    o[j] = __float_as_uint(__uint_as_float(o[j]) * f0);
                if constexpr (kKeySplit) {
                    // (the second block's columns of the same lanes; nothing there without its tiles)
                    uint32_t w[32];
                    tmem_ld32(to + kTmBlock + kTmO + 32 * cb, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (w1 != 0.f)
                            o[j] = __float_as_uint(fmaf(__uint_as_float(w[j]), f1, __uint_as_float(o[j])));
                }
                if (!has_row)
                    continue;
                if (f32) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        store_sector(dst + 128 * cb + 32 * k, wide, o[8 * k], o[8 * k + 1], o[8 * k + 2], o[8 * k + 3],
                                     o[8 * k + 4], o[8 * k + 5], o[8 * k + 6], o[8 * k + 7]);
                } else {
                    uint32_t h[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const __nv_bfloat162 two =
                            __floats2bfloat162_rn(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
                        h[j] = *reinterpret_cast<const uint32_t *>(&two);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        store_sector(dst + 64 * cb + 32 * k, wide, h[8 * k], h[8 * k + 1], h[8 * k + 2], h[8 * k + 3],
                                     h[8 * k + 4], h[8 * k + 5], h[8 * k + 6], h[8 * k + 7]);
                }
            }
            __syncwarp();
            if (kKeySplit) {
                tc_fence_before_sync();
                warp_arrive(B(S::kFree), lane);
            }
        }
        ib += my_tiles;
        ++un;
        return ok;
        });
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == S::kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 2 * kTmBlock);
    }
}

// Joins the pieces of the units that CTA blockIdx.x began and did not end: with
// reference m_j and sum l_j of piece j, M = max_j m_j,
//   o = sum_j 2^(m_j - M) O_j / sum_j 2^(m_j - M) l_j.
// The pieces are the CTA's own second one and the first ones of the CTAs after
// it, up to the one that ends the unit.  Four channels a lane.  What bounds it is
// the chain of loads (note, sums, O): a warp takes four rows where units are in
// few pieces, one row and eight pieces at a time where few rows are in many.
template <int kRows>
constexpr int kJoinRowsOf = kRows == kRowsBlock ? 1 : 4;

template <int kRows>
__global__ void __launch_bounds__(256) paged_extend_join_kernel(const __grid_constant__ PagedExtendParams p)
{
    constexpr int kJoinRows = kJoinRowsOf<kRows>, kAhead = 8 / kJoinRows;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, first = blockIdx.x;
    const Note *notes = notes_of<kRows>(p);
    const int4 n0 = __ldcg(reinterpret_cast<const int4 *>(notes + first));       // tail, h, row0, rows
    const int c0 = __ldcg(&notes[first].c0);
    int head = first + lane < p.workers ? __ldcg(&notes[first + lane].head) : 0;
    const int rr = (blockIdx.y * 8 + (threadIdx.x >> 5)) * kJoinRows, left = n0.w - n0.z - rr;     // rows from here on
    if (!n0.x || left <= 0)
        return;
    float M[kJoinRows], den[kJoinRows];
    float4 acc[kJoinRows];
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
        M[k] = -INFINITY;
        den[k] = 0.f;
        acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    bool last = false;
    for (int j0 = first; !last && j0 < p.workers; j0 += 32) {
        // lane i: piece j0 + i, if the unit reaches that far
        const int j = j0 + lane;
        if (j0 > first)
            head = j < p.workers ? __ldcg(&notes[j].head) : 0;
        else if (lane == 0)
            head = 1;                            // the piece that begins the unit
        const unsigned stop = __ballot_sync(kFullMask, head != 1);       // 2 ends it; 0 does not occur before that
        const int n = stop ? __ffs(stop) - 1 + (__shfl_sync(kFullMask, head, __ffs(stop) - 1) == 2) : 32;
        last = stop != 0;
        const size_t piece = kPieceFloats<kRows> * (2 * static_cast<size_t>(j) + (j == first));
        float2 ml[kJoinRows];
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k)
            ml[k] = lane < n ? __ldcg(reinterpret_cast<const float2 *>(p.partials + piece + kRows * kHeadDim) + rr + k)
                             : make_float2(-INFINITY, 0.f);
        float w[kJoinRows];
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k) {
            const float m = ml[k].x, l = ml[k].y;
            float top = m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
            top = fmaxf(top, M[k]);
            const float old = M[k] == -INFINITY ? 0.f : fast_exp2(M[k] - top);
            w[k] = m == -INFINITY ? 0.f : fast_exp2(m - top);
            float add = (m == -INFINITY && l != l) ? l : w[k] * l;       // a row of NaN scores stays NaN
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                add += __shfl_xor_sync(kFullMask, add, o);
            den[k] = den[k] * old + add;
            acc[k] = make_float4(acc[k].x * old, acc[k].y * old, acc[k].z * old, acc[k].w * old);
            M[k] = top;
        }
#pragma unroll kAhead
        for (int i = 0; i < n; ++i) {
            const float4 *o = reinterpret_cast<const float4 *>(
                                  p.partials +
                                  kPieceFloats<kRows> * (2 * static_cast<size_t>(j0 + i) + (j0 + i == first)) +
                                  static_cast<size_t>(rr) * kHeadDim) + lane;
            float4 v[kJoinRows];
#pragma unroll
            for (int k = 0; k < kJoinRows; ++k)  // (rows behind the last: memory of the piece, not used)
                v[k] = __ldcg(o + k * (kHeadDim / 4));
#pragma unroll
            for (int k = 0; k < kJoinRows; ++k) {
                const float wi = __shfl_sync(kFullMask, w[k], i);
                acc[k].x += wi != 0.f ? wi * v[k].x : 0.f;
                acc[k].y += wi != 0.f ? wi * v[k].y : 0.f;
                acc[k].z += wi != 0.f ? wi * v[k].z : 0.f;
                acc[k].w += wi != 0.f ? wi * v[k].w : 0.f;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
        if (k >= left)
            break;
        const float f = den[k] > 0.f ? 1.f / den[k] : 0.f;
        float4 a = make_float4(acc[k].x * f, acc[k].y * f, acc[k].z * f, acc[k].w * f);
        if (den[k] != den[k])
            a = make_float4(den[k], den[k], den[k], den[k]);
        const int row = n0.z + rr + k, t = row / p.group;
        const int64_t at = (static_cast<int64_t>(c0 + t) * p.hq + n0.y * p.group + (row - t * p.group)) * kHeadDim;
        if (p.out_f32) {
            reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at)[lane] = a;
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
            reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at)[lane] =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        }
    }
}

} // namespace

// Whether a CTA's two blocks share their rows, how many CTAs take part and the
// bytes that their pieces take, from sizes the host knows.
ExtendShape paged_extend_shape(int64_t q_rows, int64_t max_q_len, int64_t batch, int64_t hkv, int64_t group,
                               int64_t max_pages, int64_t window)
{
    ExtendShape s;
    if (max_q_len > q_rows)
        max_q_len = q_rows;                      // no chunk is longer
    s.key_split = max_q_len * group <= kRowsBlock;
    const int64_t rows = s.key_split ? kRowsBlock : 2 * kRowsBlock;
    const int64_t row_tiles = (max_q_len * group + rows - 1) / rows;
    const int64_t most = batch * row_tiles, filled = q_rows * group / rows + batch;
    int64_t keys = max_pages * kPageSize;
    if (window > 0 && window + max_q_len < keys)
        keys = window + max_q_len;
    // (the CTAs see the true lengths and leave out those that would have less
    // than kMinRun tiles)
    const int64_t sms = sm_count() > 0 ? sm_count() : 1;
    const int64_t unit = (keys + kKeys - 1) / kKeys + 1 + kUnitCost;
    // (may pass 64 bits)
    const double runs = static_cast<double>(hkv) * (most < filled ? most : filled) * unit / kMinRun;
    s.workers = runs < 1 ? 1 : (runs < sms ? static_cast<int>(runs) : static_cast<int>(sms));
    const size_t piece = (s.key_split ? kPieceFloats<kRowsBlock> : kPieceFloats<2 * kRowsBlock>)*sizeof(float);
    // No unit is cut, and there is nothing to join, where none has more than
    // kWhole tiles.
    int64_t tiles = (max_pages * kPageSize + kKeys - 1) / kKeys;
    if (window > 0) {
        // the keys of a row tile's tokens begin anywhere in a key tile
        const int64_t span = window + (max_q_len < rows / group + 2 ? max_q_len : rows / group + 2);
        const int64_t most_tiles = (span + kKeys - 1) / kKeys + 1;
        tiles = most_tiles < tiles ? most_tiles : tiles;
    }
    const bool cuts = s.workers > 1 && tiles > kWhole;
    s.workspace = cuts ? s.workers * (2 * piece + sizeof(Note)) : 0;
    return s;
}

template <bool kKeySplit>
static cudaError_t launch_extend(const PagedExtendParams &p, cudaStream_t s)
{
    using S = Shape<kKeySplit>;
    cudaError_t e = cudaFuncSetAttribute(paged_extend_kernel<kKeySplit>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         S::kSmem);
    if (e != cudaSuccess)
        return e;
    e = launch_pdl(paged_extend_kernel<kKeySplit>, dim3(p.workers), dim3(S::kThreads), S::kSmem, s, p);
    if (e != cudaSuccess || p.partials == nullptr)
        return e;
    return launch_pdl(paged_extend_join_kernel<S::kRows>,
                      dim3(p.workers - 1, S::kRows / (8 * kJoinRowsOf<S::kRows>)), dim3(256), 0, s, p);
}

cudaError_t launch_paged_extend(const PagedExtendParams &in, const ExtendShape &shape, cudaStream_t s)
{
    PagedExtendParams p = in;
    p.workers = shape.workers;
    if (shape.workspace == 0)
        p.partials = nullptr;                    // no pieces
    return shape.key_split ? launch_extend<true>(p, s) : launch_extend<false>(p, s);
}

} // namespace nvfp4kv
