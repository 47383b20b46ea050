// Decode over few pages a query token, listed or all, in one launch: a cluster of
// CTAs for each (query token, kv head).
//
// The worker split of decode_kernel balances any lengths, at the price of
// partials in the workspace and a second kernel.  Where a query token has few
// pages -- a page list, or a short sequence -- those fixed costs are most of the
// time.  Here the 8 warps of each of the cluster's 1 to 8 CTAs take equal runs of
// the pages (staged and multiplied as in decode_kernel), the warps' softmax
// states meet in shared memory and the CTAs' in the cluster's (a row's states are sent
// to the CTA that finishes it):
//   M = max_w m_w,  o = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w.
// No partial goes to memory.  Two CTAs to an SM, so that one's merge runs beside
// the other's loads.
#include "cluster.cuh"
#include "decode_common.cuh"

namespace nvfp4kv {
namespace {

constexpr int kClWarps = 8, kClThreads = 32 * kClWarps;
constexpr int kRowFloats = kHeadDim + 4;         // (rows 2tig of four lanes in different banks)
constexpr int kStateFloats = kMaxGroup * kRowFloats + 2 * kMaxGroup;

template <class Fmt>
constexpr int kClStages = Fmt::kRecord > 4000 ? 3 : 5;

// Rows that a CTA is sent to be joined, at most: r ranks * ceil(8 / r) of them.
constexpr int kSentRows = 14;

template <class Fmt>
constexpr size_t kClSmem = 128 + static_cast<size_t>(kClWarps) * kClStages<Fmt> * (Fmt::kRecord + 8 + 4) +
                           kSentRows * kRowFloats * sizeof(float);

template <class Fmt>
constexpr bool kClFits = 2 * (kClSmem<Fmt> + 1024) <= 228 * 1024 &&
                         kClStages<Fmt> *Fmt::kRecord >= kStateFloats * static_cast<int>(sizeof(float));
static_assert(kClFits<Nvfp4Format> && kClFits<Fp8BlockFormat>, "two CTAs an SM; a warp's state in its ring");

__device__ __forceinline__ float query_scale(const ClusterParams &p, int)
{
    return p.qscale;
}

__device__ __forceinline__ float query_scale(const ClusterHeadParams &p, int h)
{
    return p.qs[h];
}

template <class Fmt, bool kListed, class Params>
__global__ void __launch_bounds__(kClThreads, 2) cluster_decode_kernel(const __grid_constant__ Params p)
{
    constexpr bool kHeadScales = std::is_same_v<Params, ClusterHeadParams>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
    constexpr int S = kClStages<Fmt>, R = Fmt::kRecord;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, tig = lane & 3;
    uint8_t *ring = smem + warp * S * R;
    const uint32_t wdata = smem_addr(ring);
    const uint32_t wbar = smem_addr(smem + kClWarps * S * R) + warp * S * 8;
    // tokens of the page in each stage that count
    volatile int32_t *counted = reinterpret_cast<int32_t *>(smem + kClWarps * S * (R + 8)) + warp * S;
    // the cluster's rows that this CTA finishes, as their CTAs send them: 128 channels, M, l
    float *sent = reinterpret_cast<float *>(smem + kClWarps * S * (R + 12));

    if (lane == 0) {
        for (int s = 0; s < S; ++s)
            mbar_init(wbar + 8 * s, 1);
        fence_mbar_init();
    }
    pdl_launch_dependents();
    // Lengths and block tables may be read ahead of the kernel before, as in
    // decode_kernel; lists, queries and records may not.
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    if (ranks > 1)
        cluster_arrive();                        // (this CTA runs: it can be written to)
    const int seg = p.seg0 + blockIdx.x / ranks, row = seg / p.hkv, h = seg - row * p.hkv;
    const int b = row / p.sel_q_len;
    if (rank == 0 && h == 0 && threadIdx.x == 0 && row == b * p.sel_q_len) {
        const int L = __ldg(p.seq_lens + b);
        if (L < 0 || L > p.max_pages * kPageSize)
            report(p.dev_status, NVFP4KV_DEV_BAD_LEN);
    }
    const int sees = clamp_len(__ldg(p.seq_lens + b), p.max_pages * kPageSize) - p.sel_q_len + (row - b * p.sel_q_len) + 1;
    const int L = max(sees, 0);
    const int pages = (L + kPageSize - 1) / kPageSize, n = kListed ? min(p.budget, pages) : pages;
    const int w = rank * kClWarps + warp, workers = ranks * kClWarps;
    const int lo = static_cast<int>(static_cast<long long>(n) * w / workers);
    const int hi = static_cast<int>(static_cast<long long>(n) * (w + 1) / workers);
    const int32_t *list = kListed ? p.sel_pages + (static_cast<size_t>(row) * p.hkv + h) * p.budget : nullptr;
    const int32_t *table = p.block_table + static_cast<size_t>(b) * p.max_pages;

    // Lane l looks up entry win + l of the current window of 32, and of the next.
    uint32_t cur_rec = 0, nxt_rec = 0;
    int cur_counted = 0, nxt_counted = 0, win = lo;
    auto lookup = [&](int j) {
        nxt_rec = 0;
        nxt_counted = 0;
        if (j >= hi)
            return;
        const int page = kListed ? __ldcg(list + j) : j;
        if (page < 0 || page >= pages) {
            report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);              // (no token of it counts)
            return;
        }
        int phys = __ldg(table + page);
        if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_pages)) {
            report(p.dev_status, NVFP4KV_DEV_BAD_PAGE);
            phys = 0;
        }
        nxt_counted = min(L - page * kPageSize, kPageSize);
        nxt_rec = static_cast<uint32_t>(phys) * static_cast<uint32_t>(p.hkv) + static_cast<uint32_t>(h);
    };
    auto issue = [&](int j, int st) {
        int rel = j - win;
        if (rel >= 32) {
            win += 32;
            rel -= 32;
            cur_rec = nxt_rec;
            cur_counted = nxt_counted;
            lookup(win + 32 + lane);
        }
        const uint32_t z = __shfl_sync(kFullMask, cur_rec, rel);
        if (lane == rel)
            counted[st] = cur_counted;
        if (lane == 0) {
            const uint32_t bar = wbar + 8 * st;
            mbar_arrive_expect_tx(bar, R);
            bulk_g2s(wdata + st * R, p.pool + static_cast<size_t>(z) * R, R, bar);
        }
    };
    if (kListed)
        pdl_wait();
    lookup(lo + lane);
    cur_rec = nxt_rec;
    cur_counted = nxt_counted;
    lookup(lo + 32 + lane);
    if (!kListed)
        pdl_wait();
    for (int x = lo; x < min(lo + S, hi); ++x)
        issue(x, x - lo);

    uint32_t qf[16];
    float inv0 = 1.f, inv1 = 1.f, m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float oacc[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            oacc[j][e] = 0.f;
    {
        const bool has_row = gid < p.group;
        const uint16_t *q = p.q + (static_cast<size_t>(row) * p.hq + h * p.group + (has_row ? gid : 0)) * kHeadDim;
        if constexpr (Fmt::kPageScales)
            load_rows_apart(q, has_row, p.qscale, tig, qf, inv0, inv1);
        else
            load_rows(q, has_row ? query_scale(p, h) : 0.f, tig, qf);
    }
    const LaneOffsets off = Fmt::offsets(gid, tig);

    int st = 0;
    uint32_t ph = 0;
    for (int j = lo; j < hi;) {
        const int np = j + 1 < hi ? 2 : 1;
        int st1 = st + 1;
        uint32_t ph1 = ph;
        if (st1 == S) {
            st1 = 0;
            ph1 ^= 1u;
        }
        const bool arrived = np == 2 ? mbar_wait2_bounded(wbar + 8 * st, ph, wbar + 8 * st1, ph1, p.wait_limit)
                                     : mbar_wait_bounded(wbar + 8 * st, ph, p.wait_limit);
        if (!__all_sync(kFullMask, arrived)) {
            // staged data never arrived: report, let the copies in flight land, and
            // go to the cluster's barriers with nothing
            if (lane == 0)
                report(p.dev_status, NVFP4KV_DEV_TIMEOUT);
            for (int k = 0; k < min(S, hi - j); ++k) {
                const int s2 = st + k;
                mbar_wait_bounded(wbar + 8 * (s2 < S ? s2 : s2 - S), s2 < S ? ph : ph ^ 1u, kWaitLimit);
            }
            break;
        }
        __syncwarp();
        const int v0 = counted[st], v1 = np == 2 ? counted[st1] : v0;
        if (np == 2)
            attend_pages<Fmt, 2, Counted::kEach>(qf, inv0, inv1, m0, m1, l0, l1, oacc, wdata + st * R, wdata + st1 * R, v0,
                                                 v1, 0, 0, 0, off, gid, tig);
        else
            attend_pages<Fmt, 1, Counted::kEach>(qf, inv0, inv1, m0, m1, l0, l1, oacc, wdata + st * R, wdata + st * R, v0,
                                                 v0, 0, 0, 0, off, gid, tig);
        __syncwarp();
        if (j + S < hi)
            issue(j + S, st);
        if (np == 2 && j + 1 + S < hi)
            issue(j + 1 + S, st1);
        st += np;
        if (st >= S) {
            st -= S;
            ph ^= 1u;
        }
        j += np;
    }

    // the warp's state into its ring, whose copies have all landed
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(kFullMask, l0, o);
        l1 += __shfl_xor_sync(kFullMask, l1, o);
    }
    float *mine = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float *dst = mine + (2 * tig + which) * kRowFloats;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dst[Fmt::channel(j, gid, 0)] = oacc[j][which];
            dst[Fmt::channel(j, gid, 1)] = oacc[j][2 + which];
        }
    }
    if (gid == 0) {
        float *ml = mine + kMaxGroup * kRowFloats;
        ml[2 * tig] = m0;
        ml[2 * tig + 1] = m1;
        ml[kMaxGroup + 2 * tig] = l0;
        ml[kMaxGroup + 2 * tig + 1] = l1;
    }
    __syncthreads();
    // warp r joins row r of the CTA's warps, four channels a lane
    const int r = warp;
    constexpr int kStep = S * R / static_cast<int>(sizeof(float));   // from one warp's state to the next
    float *all = reinterpret_cast<float *>(smem);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, l = 0.f;
    if (r < p.group) {
#pragma unroll
        for (int k = 0; k < kClWarps; ++k)
            M = fmaxf(M, all[k * kStep + kMaxGroup * kRowFloats + r]);
#pragma unroll
        for (int k = 0; k < kClWarps; ++k) {
            const float *from = all + k * kStep;
            const float m = from[kMaxGroup * kRowFloats + r], e = m == -INFINITY ? 0.f : fast_exp2(m - M);
            const float4 v = *reinterpret_cast<const float4 *>(from + r * kRowFloats + 4 * lane);
            o.x += e * v.x;
            o.y += e * v.y;
            o.z += e * v.z;
            o.w += e * v.w;
            l += e * from[kMaxGroup * kRowFloats + kMaxGroup + r];
        }
    }
    if (ranks > 1) {
        // CTA r mod ranks finishes row r; sent rather than fetched, so that there is one
        // trip and nobody has to stay for the others
        const uint32_t each = (kMaxGroup + ranks - 1) / ranks;
        cluster_wait();
        if (r < p.group) {
            const uint32_t at = in_cta(smem_addr(sent + (rank * each + r / ranks) * kRowFloats), r % ranks);
            st_cluster4(at + 16 * lane, o);
            if (lane == 0)
                st_cluster4(at + 4 * kHeadDim, make_float4(M, l, 0.f, 0.f));
        }
        cluster_sync();
        if (r < p.group && r % ranks == rank) {
            const float *from = sent + r / ranks * kRowFloats;
            for (uint32_t k = 0; k < ranks; ++k)
                M = fmaxf(M, from[k * each * kRowFloats + kHeadDim]);
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            l = 0.f;
            for (uint32_t k = 0; k < ranks; ++k) {
                const float *row_k = from + k * each * kRowFloats;
                const float m = row_k[kHeadDim], e = m == -INFINITY ? 0.f : fast_exp2(m - M);
                const float4 v = *reinterpret_cast<const float4 *>(row_k + 4 * lane);
                o.x += e * v.x;
                o.y += e * v.y;
                o.z += e * v.z;
                o.w += e * v.w;
                l += e * row_k[kHeadDim + 1];
            }
        }
    }
    if (r < p.group && r % ranks == rank) {
        float osc = p.out_scale;
        if constexpr (kHeadScales)
            osc = p.vs[h];
        const float by = l > 0.f ? osc / l : 0.f;
        const size_t at = (static_cast<size_t>(row) * p.hq + h * p.group + r) * kHeadDim + 4 * lane;
        if (p.out_bf16) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * by, o.y * by), y = __floats2bfloat162_rn(o.z * by, o.w * by);
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
                make_float4(o.x * by, o.y * by, o.z * by, o.w * by);
        }
    }
}

template <class Fmt, bool kListed, class Params>
cudaError_t launch(Params &c, const DecodeParams &p, const ClusterPlan &plan, cudaStream_t s)
{
    constexpr auto kernel = cluster_decode_kernel<Fmt, kListed, Params>;
    cudaError_t e = allow_shared<kernel>();
    const int segments = p.batch * p.hkv;
    auto part = [&](int n, int ranks) {
        if (e == cudaSuccess && n > 0)
            e = launch_cluster(kernel, dim3(static_cast<unsigned>(n) * ranks), dim3(kClThreads), ranks, kClSmem<Fmt>, s, c);
        c.seg0 += n;
    };
    part(plan.first, plan.ranks);
    part(segments - plan.first, plan.rest_ranks);
    return e;
}

ClusterParams cluster_params(const DecodeParams &p)
{
    return {p.pool,      p.q,         p.out,    p.block_table, p.seq_lens, p.sel_pages, p.dev_status, p.hq,         p.hkv,
            p.group,     p.max_pages, p.num_pages, p.budget,   p.sel_q_len, p.out_bf16, p.qscale,     p.out_scale,
            p.wait_limit, 0};
}

// What plan_cluster_decode reckons with.
struct ClusterCost {
    int64_t pages, sms, slots;
    double busy, idle;           // us a page of a CTA, with a neighbour on the SM and without

    // CTAs a cluster
    int64_t ranks(int64_t segments) const
    {
        int64_t r = slots / segments;
        r = r < 8 ? r : 8;
        while ((r > 4 && segments * r > slots * 3 / 4) || (r > 2 && segments * r > slots * 6 / 7))
            --r;
        r = r < pages / kClWarps ? r : pages / kClWarps;
        return r < 1 ? 1 : r;
    }
    double wave(int64_t r, bool crowded) const { return 3.6 + (crowded ? busy : idle) * ((pages + r - 1) / r); }
    double all(int64_t segments, int64_t r) const
    {
        const int64_t full = segments * r / slots, rest = segments * r % slots;
        return full * wave(r, true) + (rest == 0 ? 0.0 : wave(r, rest > sms || r > 4));
    }
};

} // namespace

// CTAs a cluster: as many as fill two places an SM (or one place for each page and
// warp), and whether that is faster than the worker split.  Clusters of more than two
// leave some places free: their CTAs start in one part of the GPU, and where the kernel
// before leaves its SMs one by one, the last clusters wait for a part with room (a
// selection and the decode of 96 rows of 128 pages in 8 bits: 38.6 us with three CTAs a
// cluster in 288 of 304 places, 31.9 with two; 48 rows: 31.3 with six in 288, 24.5 with
// four in 192; 64 rows: 28.3 with three in 192, 27.9 with four in 256).  Full waves of one
// or two CTAs a list may leave a rest that goes faster by a launch of its own, as larger
// clusters (320 lists of 128 pages in 8 bits: 42 us by one launch, 37 by two).  Not so
// where all pages are read, whose numbers differ: the second launch cannot fill in
// behind the short ones of the first (four tokens of 12 sequences in 8 bits, all of 8K
// tokens, 97 and 85 us; of 100 to 8K, 62 and 80).
// In us, measured: a wave of clusters 3.6 and for each page of a CTA 0.115 with a
// neighbour on the SM, 0.075 without (8 bits: 0.19, or 0.105 where query tokens share
// their pages, and 0.085), a second launch 4; the workers 8.5 (8 bits: 16, or 18 for
// several tokens; their CTAs leave no registers for the next kernel's), 0.00036 (one
// token in 8 bits 0.00053) a page-head and 0.012 (0.015) a segment to be joined, of
// which `worker_segments` are row groups of up to eight query rows.  80 of 256 pages in 4
// bits: 11 and 18 us; 312 of 256: 55 and 42.  Four tokens in 8 bits: 20 sequences of 2K
// and three tokens 36 and 44, 12 of 8K 98 and 90, six of 128K to 160K 1,059 and 467.
ClusterPlan plan_cluster_decode(int64_t segments, int64_t worker_segments, int64_t pages, bool eight_bits, bool listed,
                                int q_len)
{
    const int64_t sms = sm_count();
    // (no device: the worker split's launch says so)
    if (segments < 1 || segments > (int64_t{1} << 27) || sms < 1)
        return {};
    const bool shared = !listed && q_len > 1;
    const ClusterCost cost{pages, sms, 2 * sms, eight_bits ? (shared ? 0.105 : 0.19) : 0.115, eight_bits ? 0.085 : 0.075};
    int64_t ranks = cost.ranks(segments), first = segments, rest_ranks = 1;
    double best = cost.all(segments, ranks);
    for (int64_t r = 1; listed && r <= 2 && (r == 1 || pages >= 2 * kClWarps); ++r) {
        const int64_t n = segments * r / cost.slots * (cost.slots / r), rest = segments - n;
        if (n <= 0 || rest <= 0 || cost.ranks(rest) == r)
            continue;
        const double both = cost.all(n, r) + cost.all(rest, cost.ranks(rest)) + 4.0;
        if (both < best) {
            best = both;
            ranks = r;
            first = n;
            rest_ranks = cost.ranks(rest);
        }
    }
    const double heads = static_cast<double>(worker_segments) * pages, joins = static_cast<double>(worker_segments);
    const double workers = !eight_bits ? 8.5 + 0.00036 * heads + 0.012 * joins
                           : shared    ? 18.0 + 0.00036 * heads + 0.012 * joins
                                       : 16.0 + 0.00053 * heads + 0.015 * joins;
    if (best > workers)
        return {};
    return {static_cast<int>(first), static_cast<int>(ranks), static_cast<int>(rest_ranks)};
}

cudaError_t launch_cluster_decode_nvfp4(const DecodeParams &p, const ClusterPlan &plan, cudaStream_t s)
{
    ClusterParams all = cluster_params(p);
    if (!p.hs.per_head)
        return launch<Nvfp4Format, true>(all, p, plan, s);
    ClusterHeadParams c{all, {}, {}};
    for (int h = 0; h < p.hkv; ++h) {
        c.qs[h] = p.qs[h];
        c.vs[h] = p.hs.v[h];
    }
    return launch<Nvfp4Format, true>(c, p, plan, s);
}

cudaError_t launch_cluster_decode_fp8_block(const DecodeParams &p, const ClusterPlan &plan, cudaStream_t s)
{
    ClusterParams c = cluster_params(p);
    return p.sel_pages != nullptr ? launch<Fp8BlockFormat, true>(c, p, plan, s) : launch<Fp8BlockFormat, false>(c, p, plan, s);
}

} // namespace nvfp4kv
