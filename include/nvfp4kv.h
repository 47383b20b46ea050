/*
 * nvfp4kv -- NVFP4 paged KV cache for GQA decode on one GB300 (sm_103a).
 *
 * C ABI.  Plain pointers and sizes only.  Every device pointer is a CUDA
 * device address owned by the caller; the library allocates no device memory
 * and keeps no state between calls except a per-device cache of the SM count
 * and the fixed scratch array of nvfp4kv_paged_decode_static_scratch.
 * Every launching call is asynchronous on the given stream: it validates its
 * arguments on the host first (returning an error and launching nothing when
 * they are bad), then enqueues its kernels and returns.  A NULL stream is the
 * legacy default stream.
 *
 * The method (from the pages this library implements; cited by title and
 * section):
 *   "SGLang stores KV cache in 4 bits: long-context decode throughput rises
 *   26-30%, ..." (summary of the LMSYS post "Accelerating Long-Context and
 *   Agentic Inference with NVFP4 KV Cache"), Interpretation: the KV cache is
 *   paged; each block of 16 values is 8 bytes of packed 4-bit data plus one
 *   byte of block scale; decode dequantises inside the attention kernel; the
 *   extend path dequantises the cached prefix into an FP8 workspace; prefill
 *   quantises the new K/V into the cache.  Perspective: the per-tensor FP32
 *   global scale is left at 1.0.
 *   "NVFP4-KV-Cache auf der NVIDIA RTX PRO 6000 Blackwell Server Edition",
 *   "Bytes pro Token": E2M1 elements (1 sign, 2 exponent, 1 mantissa bit),
 *   one FP8-E4M3 scale per 16 values, an FP32 tensor scale above them;
 *   "Unterstuetzung in den Engines": the FP8-E4M3 cache is the baseline.
 *
 * Formats (readings where the pages are silent):
 *   E2M1 code: bit 3 sign, bits 2..1 exponent (bias 1), bit 0 mantissa;
 *     magnitudes {0, 0.5, 1, 1.5, 2, 3, 4, 6}.
 *   E4M3 (OCP "FN"): bias 7, subnormals m/8 * 2^-6, max 448, 0x7F = NaN.
 *   Tensor scale G (nvfp4kv_cache.global_scale, FP32; the pages run with
 *     G = 1.0 and name its calibration as the next step): a cached value is
 *     G * E4M3 block scale * E2M1 code.
 *   Block of 16 consecutive channels of one token-head, y_i = fl32(x_i / G)
 *     (y = x at G = 1):
 *     S = E4M3_rn_satfinite(fl32(amax_i |y_i| / 6)), s = value(S),
 *     q_i = E2M1_rn_satfinite(fl32(y_i / s)), or 0 for all i if s == 0.
 *     Packed byte j = q_{2j} | q_{2j+1} << 4 (low nibble = even channel).
 *
 * Cache layout.  The cache is one pool of page-head records: the record of
 * kv head h of physical page P starts at byte (P * num_kv_heads + h) * R and
 * holds the 16 tokens of that page for that head (token t of the page is the
 * one at slot P * 16 + t).  The pages give only the storage cost (8 packed
 * bytes + 1 scale byte per 16 values); the arrangement inside a record is this
 * library's, chosen so the decode stages a record with one bulk copy and reads
 * it without shared-memory bank conflicts.
 *
 * NVFP4 record, R = NVFP4KV_RECORD_BYTES = 2304:
 *   [0, 1024)     K data: 16 rows of 64 bytes, row t = token t; byte 8*b + i
 *                 of a row holds channels 16*b + 2i (low nibble) and
 *                 16*b + 2i + 1 (high nibble).
 *   [1024, 2048)  V data: 8 rows of 128 bytes; row p holds tokens 2p (low
 *                 nibbles) and 2p + 1 (high nibbles) of the same channel.  A row
 *                 is 8 chunks of 16 bytes; group g (0..7) sits in the chunk at
 *                 position (g + 2p) mod 8, and byte 2j + w of group g is
 *                 channel 16j + g + 8w.
 *   [2048, 2176)  K scales: [16 tokens][8 blocks] E4M3 (block b = channels
 *                 16b .. 16b + 15).
 *   [2176, 2304)  V scales: [8 rows p][8 blocks][2]; byte (p, b, w) is the scale
 *                 of token 2p + w, block b.
 * FP8 record, R = FP8KV_RECORD_BYTES = 4096 (E4M3 at scale 1.0):
 *   [0, 2048)     K: 16 rows of 128 bytes, row t = token t; the 16-byte chunk
 *                 at position (c + (t mod 2)) mod 8
 *                 holds channels 16c .. 16c + 15.
 *   [2048, 4096)  V: 8 rows of 256 bytes, row p = tokens 2p and 2p + 1; the
 *                 16-byte chunk at position (c + f(p)) mod 16, with
 *                 f(p) = (p mod 2) + 4 * (floor(p / 2) mod 2), holds channels
 *                 8c .. 8c + 7, byte 2i + w being channel 8c + i of token 2p + w.
 *
 * Block-scaled FP8 record, R = FP8BKV_RECORD_BYTES = 4128: the FP8 record, with
 *   codes relative to a scale, and behind it the scales of its page-head, fp32
 *   powers of two:
 *   [4096, 4100)  K scale; [4100, 4104) V scale; [4104, 4128) not used.
 *
 * Supported geometry: head_dim 128, page_size 16, num_q_heads a multiple of
 * num_kv_heads with group g = num_q_heads / num_kv_heads in 1..8,
 * global_scale a positive normal finite fp32.  Anything else returns
 * NVFP4KV_ERR_UNSUPPORTED.
 *
 * Device-side checks: kernels that read page ids, slots or lengths from
 * device memory check them and, instead of faulting, OR a bit into the
 * optional caller-owned device word *dev_status (int32, may be NULL) and
 * treat the item as described per call.  Read it after synchronising.
 */
#ifndef NVFP4KV_H
#define NVFP4KV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque CUDA stream handle (the same object as cudaStream_t). */
typedef struct CUstream_st *nvfp4kv_stream_t;

typedef enum {
    NVFP4KV_OK = 0,
    NVFP4KV_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, negative size ... */
    NVFP4KV_ERR_UNSUPPORTED = 2,  /* valid but outside the supported geometry   */
    NVFP4KV_ERR_WORKSPACE = 3,    /* decode workspace smaller than required     */
    NVFP4KV_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed       */
    NVFP4KV_ERR_DEVICE_CHECK = 5  /* a kernel set bits in the device status word */
} nvfp4kv_status;

/* Bits ORed into *dev_status by the kernels. */
#define NVFP4KV_DEV_BAD_PAGE 0x1  /* block-table entry outside [0, num_pages)     */
#define NVFP4KV_DEV_BAD_SLOT 0x2  /* slot outside [0, num_pages * page_size)      */
#define NVFP4KV_DEV_BAD_LEN 0x4   /* length < 0 or > max_pages_per_seq*page_size  */
#define NVFP4KV_DEV_TIMEOUT 0x8   /* a bounded wait for staged data gave up        */
#define NVFP4KV_DEV_NO_PAGES 0x10 /* a step needs more pages than are free         */

/* Element types of caller buffers.  NVFP4KV_E4M3 (OCP FP8 E4M3FN bytes at
 * scale 1.0) is accepted only where a call says so: the chunk K/V of the
 * extend calls. */
typedef enum { NVFP4KV_F32 = 0, NVFP4KV_BF16 = 1, NVFP4KV_E4M3 = 2 } nvfp4kv_dtype;

#define NVFP4KV_RECORD_BYTES 2304
#define FP8KV_RECORD_BYTES 4096
#define FP8BKV_RECORD_BYTES 4128

/* NVFP4 cache: pool of num_pages * num_kv_heads records laid out as above,
 * 16-byte aligned; global_scale is the tensor scale G described above.
 * head_scales (optional, may be NULL): a HOST array of 2 * num_kv_heads
 * per-head factors, K then V.  With it, kv head h of K uses the tensor scale
 * G_h = fl32(global_scale * head_scales[h]) and of V fl32(global_scale *
 * head_scales[num_kv_heads + h]) wherever G appears above (a refinement of the
 * pages' single tensor scale; this library's).  Each factor and each product
 * must be a positive normal finite float, and num_kv_heads at most
 * NVFP4KV_MAX_SCALED_KV_HEADS, else calls return NVFP4KV_ERR_UNSUPPORTED.  The
 * values are read on the host during each call. */
#define NVFP4KV_MAX_SCALED_KV_HEADS 128

typedef struct {
    void *pool;
    int32_t num_pages;
    int32_t num_kv_heads;
    int32_t page_size;
    int32_t head_dim;
    float global_scale;
    const float *head_scales;
} nvfp4kv_cache;

/* FP8-E4M3 comparison cache (scale 1.0): pool of records as above, 16-byte
 * aligned. */
typedef struct {
    void *pool;
    int32_t num_pages;
    int32_t num_kv_heads;
    int32_t page_size;
    int32_t head_dim;
} fp8kv_cache;

/* FP8-E4M3 cache with a scale for each page and kv head: pool of records as
 * above, 16-byte aligned. */
typedef struct {
    void *pool;
    int32_t num_pages;
    int32_t num_kv_heads;
    int32_t page_size;
    int32_t head_dim;
} fp8bkv_cache;

/* Bounds of the keys of each page and kv head (see nvfp4kv_page_bounds):
 * bounds int8 [num_pages][num_kv_heads][2][128], 16-byte aligned, and steps fp32
 * [num_pages][num_kv_heads].  They belong to one cache: its page ids, its heads. */
typedef struct {
    int8_t *bounds;
    float *steps;
    int32_t num_pages;
    int32_t num_kv_heads;
} nvfp4kv_bounds;

/* Write side ("SGLang stores KV cache in 4 bits", Interpretation ¶2: prefill
 * quantises the new K/V into the NVFP4 cache).
 * k_new, v_new: [num_tokens][num_kv_heads][head_dim] contiguous, fp32 or bf16
 *   (in_dtype), 16-byte aligned; read only.
 * slot_mapping: int32[num_tokens] device array; slot < 0 skips the token; a
 *   slot >= num_pages * page_size is skipped and sets NVFP4KV_DEV_BAD_SLOT.
 *   Slots must be distinct (two tokens writing one slot is a data race).
 * Writes the data and scale bytes of every (token, kv head) row of K and V.
 * Inputs must be finite (non-finite values give unspecified codes). */
nvfp4kv_status nvfp4kv_quantize_append(const nvfp4kv_cache *cache, const void *k_new,
                                       const void *v_new, nvfp4kv_dtype in_dtype,
                                       int32_t num_tokens, const int32_t *slot_mapping,
                                       int32_t *dev_status, nvfp4kv_stream_t stream);

/* Largest batch one decode call takes (the per-sequence page-head offsets are
 * kept in shared memory next to the staging ring); a larger batch returns
 * NVFP4KV_ERR_UNSUPPORTED. */
#define NVFP4KV_MAX_BATCH 8192

/* Bytes of decode workspace needed by nvfp4kv_paged_decode / fp8kv_paged_decode
 * when called with the same num_workers on the current device (num_workers 0 =
 * the automatic choice, whose need is bounded by this value).  Host only; the
 * result depends on the current device's SM count.  A library utility: the
 * pages describe no workspace (the split-KV scratch is this library's
 * design). */
size_t nvfp4kv_decode_workspace_size(int32_t num_workers);

/* Decode attention over the NVFP4 cache ("SGLang stores KV cache in 4 bits",
 * Interpretation ¶2: the decode path dequantises inside the attention kernel;
 * "NVFP4-KV-Cache auf der ...", "Geschwindigkeit": bf16 queries against
 * NVFP4 keys and values).
 * For sequence b and query head i (kv head h = i / g):
 *   o[b][i] = sum_j softmax_j(sm_scale * q[b][i] . k_j) v_j over the
 *   seq_lens[b] tokens j of sequence b, token j in page block_table[b][j/16]
 *   at offset j%16; no causal mask (the query sees all cached tokens).
 * q: bf16 [batch][num_q_heads][128], 16-byte aligned.  Computation: q is
 *   multiplied by sm_scale*log2(e)*G (G the tensor scale) and rounded to fp16
 *   (|q * sm_scale * G| must stay below 4.5e4); K and V are dequantised
 *   exactly to fp16 (block scale times code) and the output is multiplied by
 *   G; QK^T and PV run
 *   on tensor cores with fp32 accumulation; softmax in fp32.
 * block_table: int32 [batch][max_pages_per_seq]; only the first
 *   ceil(seq_lens[b]/16) entries of row b are read; an entry outside
 *   [0, num_pages) reads page 0 instead and sets NVFP4KV_DEV_BAD_PAGE.
 * seq_lens: int32[batch]; a length outside [0, max_pages_per_seq*16] is
 *   clamped into it and sets NVFP4KV_DEV_BAD_LEN.  Length 0 gives zeros.
 * out: [batch][num_q_heads][128] in out_dtype, 16-byte aligned.
 * workspace: device scratch of workspace_bytes >= the size above, 256-byte
 *   aligned; its contents need no initialisation and are overwritten.  Two
 *   calls in flight at once must not share a workspace.
 * num_workers: 0 = automatic; otherwise the number of warp workers the
 *   page-heads are balanced over (results agree up to rounding for any
 *   value).
 * Launches two kernels (split-KV attention, then the split merge), both with
 * programmatic dependent launch allowed, so each may start its prologue while
 * the previous kernel in the stream drains.  seq_lens and block_table are read
 * in that prologue: a kernel earlier in the stream that writes them must not
 * let its dependents start before it has written them (no kernel of this
 * library writes them). */
nvfp4kv_status nvfp4kv_paged_decode(const nvfp4kv_cache *cache, const void *q,
                                    int32_t batch, int32_t num_q_heads,
                                    const int32_t *block_table, int32_t max_pages_per_seq,
                                    const int32_t *seq_lens, float sm_scale, void *out,
                                    nvfp4kv_dtype out_dtype, void *workspace,
                                    size_t workspace_bytes, int32_t num_workers,
                                    int32_t *dev_status, nvfp4kv_stream_t stream);

/* One decode step: append each sequence's newest token, then attend
 * ("SGLang stores KV cache in 4 bits", Interpretation: new K/V are written to
 * the cache in NVFP4 and the decode path dequantises inside attention; doing
 * both in one launch is this library's fusion, not described on the pages).
 * For every sequence b with seq_lens[b] > 0, the K and V rows k_new[b],
 * v_new[b] ([batch][num_kv_heads][128], fp32 or bf16 per in_dtype, 16-byte
 * aligned) are quantised into the cache at position seq_lens[b] - 1 (page
 * block_table[b][(seq_lens[b]-1)/16], offset (seq_lens[b]-1)%16) exactly as
 * nvfp4kv_quantize_append would, and then the decode of nvfp4kv_paged_decode
 * runs over all seq_lens[b] tokens, including the new one.  The append is done
 * inside the decode kernel by the warp that streams that page, so the step is
 * two kernels instead of three.  The page that receives a sequence's new
 * token must not appear in another sequence's block table in the same call.
 * Other arguments and results as for nvfp4kv_paged_decode. */
nvfp4kv_status nvfp4kv_append_paged_decode(const nvfp4kv_cache *cache, const void *k_new, const void *v_new,
                                           nvfp4kv_dtype in_dtype, const void *q, int32_t batch,
                                           int32_t num_q_heads, const int32_t *block_table,
                                           int32_t max_pages_per_seq, const int32_t *seq_lens, float sm_scale,
                                           void *out, nvfp4kv_dtype out_dtype, void *workspace,
                                           size_t workspace_bytes, int32_t num_workers, int32_t *dev_status,
                                           nvfp4kv_stream_t stream);

/* Multi-query decode (several new tokens per sequence at once, as in
 * multi-token prediction or speculative decoding; "NVFP4-KV-Cache auf der
 * ...", "Unterstuetzung in den Engines": the engines' NVFP4 decode paths are
 * judged on speculative decoding with multi-token prediction): q_len query tokens per
 * sequence sit at the last q_len positions and attend causally, token t
 * (0-based) over the seq_lens[b] - q_len + t + 1 first cached tokens (the
 * new tokens must already be in the cache, e.g. by nvfp4kv_quantize_append).
 * Same arguments as nvfp4kv_paged_decode except
 * q: bf16 [batch][q_len][num_q_heads][128] and out: [batch][q_len][num_q_heads]
 *   [128]; 1 <= q_len <= NVFP4KV_MAX_QUERY_TOKENS (a larger value returns
 *   NVFP4KV_ERR_UNSUPPORTED).  A query that sees no cached token gets zeros.
 * The group * q_len query rows of a kv head are processed in row groups of
 * 8; each row group streams the kv head's pages (the row groups of one kv
 * head run close together, so the repeats mostly hit L2).  The workspace is
 * sized as for nvfp4kv_paged_decode. */
#define NVFP4KV_MAX_QUERY_TOKENS 8
nvfp4kv_status nvfp4kv_paged_decode_multi(const nvfp4kv_cache *cache, const void *q, int32_t batch,
                                          int32_t q_len, int32_t num_q_heads, const int32_t *block_table,
                                          int32_t max_pages_per_seq, const int32_t *seq_lens, float sm_scale,
                                          void *out, nvfp4kv_dtype out_dtype, void *workspace,
                                          size_t workspace_bytes, int32_t num_workers, int32_t *dev_status,
                                          nvfp4kv_stream_t stream);

/* Decode without a caller-provided workspace, for callers that cannot
 * allocate device memory (for example a serving engine whose device memory is
 * all reserved for weights and KV cache at start-up).  The pages have no
 * counterpart to this call; it exists for such callers.
 * Same arguments and result as nvfp4kv_paged_decode, minus the workspace: the
 * split-KV scratch comes from one array of NVFP4KV_STATIC_SCRATCH_BYTES that
 * the library keeps on every device that loads it, until the process exits.
 * num_workers may be at most NVFP4KV_STATIC_SCRATCH_MAX_WORKERS (a larger
 * value returns NVFP4KV_ERR_WORKSPACE); 0 picks the automatic count, capped at
 * that maximum.  The first call on a device looks the array up with that
 * device current, so make it before any stream capture.  All calls on a
 * device share the array: calls whose kernels can overlap on the GPU race and
 * must be serialised (for example, issue them on one stream).  Allocates no
 * memory. */
#define NVFP4KV_STATIC_SCRATCH_BYTES (24u << 20)
#define NVFP4KV_STATIC_SCRATCH_MAX_WORKERS 3024
nvfp4kv_status nvfp4kv_paged_decode_static_scratch(const nvfp4kv_cache *cache, const void *q, int32_t batch,
                                                   int32_t num_q_heads, const int32_t *block_table,
                                                   int32_t max_pages_per_seq, const int32_t *seq_lens,
                                                   float sm_scale, void *out, nvfp4kv_dtype out_dtype,
                                                   int32_t num_workers, int32_t *dev_status,
                                                   nvfp4kv_stream_t stream);

/* Extend path ("SGLang stores KV cache in 4 bits", Interpretation ¶2: the
 * cached prefix is dequantised into one FP8 workspace shared across layers).
 * For sequence b, token j < prefix_lens[b], kv head h, channel c:
 *   out[kv_indptr[b] + j][h][c] = E4M3_rn_satfinite(fl32(E2M1 x scale x G))
 * for K into k_fp8_out and V into v_fp8_out (each [rows][num_kv_heads][128]
 * uint8, 16-byte aligned; the caller sizes it to cover every row written).
 * kv_indptr: int32[batch] row offsets; prefix_lens: int32[batch].
 * Page-id and length checks as in nvfp4kv_paged_decode. */
nvfp4kv_status nvfp4kv_dequant_prefix_fp8(const nvfp4kv_cache *cache,
                                          const int32_t *block_table,
                                          int32_t max_pages_per_seq,
                                          const int32_t *prefix_lens,
                                          const int32_t *kv_indptr, int32_t batch,
                                          void *k_fp8_out, void *v_fp8_out,
                                          int32_t *dev_status, nvfp4kv_stream_t stream);

/* Extend attention over the FP8 prefix workspace and the current chunk
 * ("SGLang stores KV cache in 4 bits", Interpretation: the extend path
 * dequantises the cached prefix into one FP8 workspace and attends over it
 * together with the new chunk).  For sequence b with chunk rows
 * [q_indptr[b], q_indptr[b+1]) and prefix length P = prefix_lens[b], chunk
 * token t (row q_indptr[b] + t) and query head i (kv head h = i / g):
 *   keys   = k_prefix[kv_indptr[b] + j][h] for j < P, then k_chunk[q_indptr[b] + u][h] for u <= t
 *   values = the same rows of v_prefix / v_chunk
 *   out[q_indptr[b] + t][i] = softmax_j(sm_scale * q . key_j) . value_j
 * Prefix keys and values are E4M3 bytes (the workspace written by
 * nvfp4kv_dequant_prefix_fp8, with the same kv_indptr and prefix_lens); q is
 * bf16; chunk keys and values are bf16 or E4M3 (chunk_dtype).  E4M3 chunk K/V
 * are initial prefill as "SGLang stores KV cache in 4 bits", Interpretation
 * ¶2 describes it: attention reads the current prompt's FP8 keys and values
 * directly (prefix length 0 there; a prefix is allowed too).
 *   q        bf16 [q_rows][num_q_heads][128]
 *   k_chunk, v_chunk  [q_rows][num_kv_heads][128], chunk_dtype NVFP4KV_BF16
 *            (bf16) or NVFP4KV_E4M3 (uint8 E4M3 codes at scale 1.0); anything
 *            else returns NVFP4KV_ERR_INVALID_ARG
 *   out      [q_rows][num_q_heads][128], out_dtype bf16 or fp32; rows outside
 *            every [q_indptr[b], q_indptr[b+1]) are not written
 *   k_prefix, v_prefix  uint8 E4M3 [prefix_rows][num_kv_heads][128]
 *   q_indptr int32 [batch + 1] (device), kv_indptr and prefix_lens int32
 *            [batch] (device)
 *   max_q_len  host bound on every q_indptr[b+1] - q_indptr[b]; it sizes the
 *            launch
 * Arithmetic.  With E4M3 chunk K/V, or bf16 ones behind prefix_rows of at
 * least 8 * q_rows: q meets the keys as two E4M3 terms of its bf16 values,
 * each row multiplied by a power of two first (exact for every element but
 * those below 2^-10 of the row's largest, whose error stays under 2^-17 of
 * it), and sm_scale * log2(e) is applied to the fp32 scores; bf16 chunk keys
 * are split the same way per 64-key tile.  Otherwise q * sm_scale * log2(e)
 * and bf16 chunk keys are rounded to fp16 (exact for bf16 values of magnitude
 * 2^-14 .. 65504; the caller keeps |q * sm_scale| below 65504).  Values: E4M3
 * to fp16 is exact, bf16 chunk values are rounded to fp16 (kept below 65504
 * by the caller).  Scores and outputs accumulate in fp32, softmax weights are
 * rounded to fp16 for the value product.
 * Pointers 16-byte aligned (index arrays 4-byte).  Group g = num_q_heads /
 * num_kv_heads in 1..8; batch and num_kv_heads at most 65535.  Device check:
 * a sequence whose q_indptr range is not inside [0, q_rows] or longer than
 * max_q_len, or whose prefix rows are not inside [0, prefix_rows), sets
 * NVFP4KV_DEV_BAD_LEN and its output rows are not written.  A sequence with
 * an empty chunk writes nothing; with an empty prefix it is causal
 * attention over the chunk alone. */
nvfp4kv_status nvfp4kv_extend_attention_fp8(const void *q, const int32_t *q_indptr, int32_t q_rows,
                                            int32_t max_q_len, const void *k_prefix,
                                            const void *v_prefix, const int32_t *kv_indptr,
                                            const int32_t *prefix_lens, int64_t prefix_rows,
                                            const void *k_chunk, const void *v_chunk,
                                            nvfp4kv_dtype chunk_dtype, int32_t batch,
                                            int32_t num_q_heads, int32_t num_kv_heads, float sm_scale,
                                            void *out, nvfp4kv_dtype out_dtype, int32_t *dev_status,
                                            nvfp4kv_stream_t stream);

/* Extend attention fused with the NVFP4 write of the chunk ("SGLang stores KV
 * cache in 4 bits", Interpretation: prefill quantises the new K/V into the
 * cache; the fusion removes the separate read of the chunk).  Computes out
 * exactly as nvfp4kv_extend_attention_fp8 (num_kv_heads taken from the cache)
 * and writes chunk row r's K and V into slot slot_mapping[r] of the cache, as
 * nvfp4kv_quantize_append would given the chunk's values (bf16 as they are;
 * E4M3 codes as the fp32 values they stand for: the same data the attention
 * reads, as initial prefill does) -- same blocks, same bytes, same tensor
 * scale; slot < 0 skips the token, a slot >= num_pages * page_size is skipped
 * and sets NVFP4KV_DEV_BAD_SLOT.  slot_mapping: int32
 * [q_rows] (device, 4-byte aligned), read only for rows inside a sequence's
 * q_indptr range; slots must be distinct.  The prefix workspace must not
 * overlap the cache. */
nvfp4kv_status nvfp4kv_extend_attention_fp8_append(const nvfp4kv_cache *cache,
                                                   const int32_t *slot_mapping, const void *q,
                                                   const int32_t *q_indptr, int32_t q_rows,
                                                   int32_t max_q_len, const void *k_prefix,
                                                   const void *v_prefix, const int32_t *kv_indptr,
                                                   const int32_t *prefix_lens, int64_t prefix_rows,
                                                   const void *k_chunk, const void *v_chunk,
                                                   nvfp4kv_dtype chunk_dtype,
                                                   int32_t batch, int32_t num_q_heads, float sm_scale,
                                                   void *out, nvfp4kv_dtype out_dtype,
                                                   int32_t *dev_status, nvfp4kv_stream_t stream);

/* Chunk attention over the paged NVFP4 cache itself ("SGLang stores KV cache in
 * 4 bits", Interpretation: attention dequantises the cached keys and values
 * inside the kernel; there for decode, here for chunks of any length: prompt
 * chunks, and drafted tokens to be checked, without the FP8 workspace, its
 * pass over the prefix and its second rounding).  The chunk's tokens are in
 * the cache already (nvfp4kv_quantize_append or nvfp4kv_qk_norm_rope_append):
 * they are the last C = q_indptr[b+1] - q_indptr[b] of the seq_lens[b] tokens of
 * sequence b, so chunk token t sits at position n = seq_lens[b] - C + t.  Query
 * head i (kv head h = i / g) attends causally:
 *   out[q_indptr[b] + t][i] = sum_j softmax_j(sm_scale * q . k_j) v_j over
 *   j = max(0, n - window + 1) .. n   (window 0: j = 0 .. n)
 * A row that sees no key (n < 0: a chunk longer than its sequence) gets zeros.
 *   q            bf16 [q_rows][num_q_heads][128]
 *   out          [q_rows][num_q_heads][128], out_dtype bf16 or fp32; rows
 *                outside every [q_indptr[b], q_indptr[b+1]) are not written
 *   q_indptr     int32 [batch + 1], seq_lens int32 [batch] (device)
 *   block_table  int32 [batch][max_pages_per_seq] (device); only entries of pages
 *                that some row sees are read, so entries that a window has left
 *                behind may hold anything; one outside [0, num_pages) reads page
 *                0 and sets NVFP4KV_DEV_BAD_PAGE
 *   max_q_len    host bound on every C; it sizes the launch
 *   window       0, or the number of keys a query sees at most, itself included
 *   workspace    device scratch of at least the size below, 256-byte aligned,
 *                not initialised (may be NULL when that is 0); two calls in
 *                flight at once must not share it
 * Pointers 16-byte aligned (index arrays 4-byte); out overlaps nothing else.
 * Group g in 1..8, batch at most NVFP4KV_MAX_BATCH, kv heads at most 65535,
 * max_q_len * g below 2^30.
 * Arithmetic: every cached value is exact in fp16, q too (bf16 significands
 * under a power of two a row; elements under 2^-28 of the row's largest lose
 * bits), scores, softmax and outputs in fp32, softmax weights rounded to fp16
 * for the value product (each off by 2^-11 of itself, and those more than 14 log2
 * units behind the row's largest by no more than 2^-10 of the row's sum of weights
 * altogether, up to 2^23 keys and scores of 2^24 log2 units).  A query with a NaN
 * or an infinity makes its row NaN if it sees a key; so may scores past fp32's range.
 * A scale byte of 0x7F, which the quantiser never writes, reads as 480.  A
 * sequence whose index range is outside [0, q_rows] or
 * longer than max_q_len, or whose length is outside [0, max_pages_per_seq *
 * 16], sets NVFP4KV_DEV_BAD_LEN and its rows are not written. */
nvfp4kv_status nvfp4kv_paged_extend(const nvfp4kv_cache *cache, const void *q, const int32_t *q_indptr,
                                    int32_t q_rows, int32_t max_q_len, int32_t batch, int32_t num_q_heads,
                                    const int32_t *block_table, int32_t max_pages_per_seq,
                                    const int32_t *seq_lens, int32_t window, float sm_scale, void *out,
                                    nvfp4kv_dtype out_dtype, void *workspace, size_t workspace_bytes,
                                    int32_t *dev_status, nvfp4kv_stream_t stream);

/* Bytes of workspace that nvfp4kv_paged_extend needs with the same sizes on the
 * current device (a library utility; 0 for sizes that the call refuses).  Host
 * only; the result depends on the current device's SM count. */
size_t nvfp4kv_paged_extend_workspace_size(int32_t q_rows, int32_t max_q_len, int32_t batch, int32_t num_q_heads,
                                           int32_t num_kv_heads, int32_t max_pages_per_seq, int32_t window);

/* ---- A step's tables, built on the device ------------------------------------
 *
 * A library utility: the pages name a paged cache ("SGLang stores KV cache in
 * 4 bits", Interpretation) and leave its bookkeeping to the engine.  These two
 * calls keep it on the device, so that a whole serving step, its page
 * allocation included, can be captured into a graph.
 *
 * Free pages are a stack: free_pages[0 .. n - 1] are the ids of the free pages
 * and *num_free = n (device int32).  plan_step takes from the top,
 * release_pages puts back on top.
 *
 * nvfp4kv_plan_step: request b has context_lens[b] cached tokens, in the pages
 * that its row of block_table lists, and adds new_lens[b] tokens (0 is
 * allowed).  With had = ceil(context / 16) and has = ceil((context + new) / 16),
 * it takes has - had fresh pages; fresh pages are numbered over the whole step
 * in the order of (request, page), and the i-th is free_pages[n - 1 - i].
 *   block_table  int32 [batch][max_pages_per_seq]: entries had .. has - 1 of
 *                row b are written, the others left as they are
 *   seq_lens     [batch]: context + new
 *   q_indptr     [batch + 1]: running sum of new_lens, from 0
 *   kv_indptr    [batch] or NULL: running sum of context_lens, from 0 (the row
 *                offsets that nvfp4kv_dequant_prefix_fp8 takes)
 *   slot_mapping [max_tokens]: row r of the step's tokens, the requests' new
 *                tokens one after another, goes to page * 16 + position mod 16;
 *                rows behind the last token get -1, which appending calls skip
 *   positions    [max_tokens] or NULL: the row's position in its sequence; -1
 *                behind the last token
 *   num_free_out the pages left, n - fresh; may be num_free_in itself
 * A request whose lengths are negative or pass max_pages_per_seq * 16 counts as
 * empty (length 0, no tokens) and sets NVFP4KV_DEV_BAD_LEN.  A page id outside
 * [0, num_pages) gives its tokens the slot -1 and sets NVFP4KV_DEV_BAD_PAGE.
 * The step is taken as a whole or not at all: if it needs more than n pages
 * (NVFP4KV_DEV_NO_PAGES), has more than max_tokens tokens, contexts that sum
 * past 2^31 - 1, or n is outside [0, free_capacity] (NVFP4KV_DEV_BAD_LEN),
 * then no page is taken, seq_lens are the context lengths, q_indptr is all 0,
 * slots and positions are -1 (kv_indptr is all 0 where its sum does not fit)
 * and num_free_out is n, clamped into that range.
 * batch at most NVFP4KV_MAX_BATCH; num_pages * 16 below 2^31.  An output must
 * not overlap another array, num_free_out on num_free_in excepted
 * (NVFP4KV_ERR_INVALID_ARG).  The decode calls read seq_lens and block_table
 * ahead of their wait for the kernel before them: this call's kernels let no
 * other kernel start before they have written both. */
nvfp4kv_status nvfp4kv_plan_step(const int32_t *context_lens, const int32_t *new_lens, int32_t batch,
                                 int32_t *block_table, int32_t max_pages_per_seq, int32_t num_pages,
                                 const int32_t *free_pages, int32_t free_capacity, const int32_t *num_free_in,
                                 int32_t *num_free_out, int32_t *seq_lens, int32_t *q_indptr, int32_t *kv_indptr,
                                 int32_t *slot_mapping, int32_t *positions, int32_t max_tokens,
                                 int32_t *dev_status, nvfp4kv_stream_t stream);

/* nvfp4kv_release_pages (a library utility): request b keeps its first
 * keep_lens[b] of old_lens[b] tokens (0: the request has ended; fewer than
 * before: drafted tokens were rejected).  Pages ceil(keep / 16) ..
 * ceil(old / 16) - 1 of its row go back: over all requests, in the order of
 * (request, page), they are written to free_pages[n], free_pages[n + 1], ...
 * and *num_free_out = n + their number (may be num_free_in itself).  The block
 * table is left as it is.  A request with keep > old, a negative length or one
 * past max_pages_per_seq * 16 returns nothing and sets NVFP4KV_DEV_BAD_LEN; a
 * page id outside [0, num_pages) goes back as it is and sets
 * NVFP4KV_DEV_BAD_PAGE.  If the stack would pass free_capacity, or n is outside
 * [0, free_capacity], nothing goes back (NVFP4KV_DEV_BAD_LEN; num_free_out is n
 * clamped into that range).  A page must be
 * held by one request only.  Limits as for nvfp4kv_plan_step. */
nvfp4kv_status nvfp4kv_release_pages(const int32_t *old_lens, const int32_t *keep_lens, int32_t batch,
                                     const int32_t *block_table, int32_t max_pages_per_seq, int32_t num_pages,
                                     int32_t *free_pages, int32_t free_capacity, const int32_t *num_free_in,
                                     int32_t *num_free_out, int32_t *dev_status, nvfp4kv_stream_t stream);

/* ---- Head norm and position rotation of new queries and keys -------------------
 *
 * The pages start from finished queries and keys; this step before the cache
 * write has no counterpart on the pages.
 *
 * For each row x of 128 channels (one token, one head) at position n:
 *   y = x / sqrt(mean(x^2) + eps) * weight              (where a norm is given)
 *   (y_a, y_b) -> scale * (y_a cos t - y_b sin t, y_b cos t + y_a sin t),
 *   t = n * inv_freq[i], for the rotary_dim / 2 channel pairs (a, b) =
 *   (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved.
 * Channels from rotary_dim on keep y.  Arithmetic in fp32, rounded once; whole
 * turns are taken off the angles in 64-bit integers, so they are as good at
 * every position as near 0. */
typedef struct {
    const double *inv_freq;      /* HOST array of rotary_dim / 2 finite values, radians a position */
    int32_t rotary_dim;          /* 0 (no rotation), 32, 64, 96 or 128 */
    int32_t interleaved;         /* 0 or 1 */
    float scale;                 /* multiplies cos and sin; finite (1 for plain rotation) */
} nvfp4kv_rope;

/* Weights: device arrays [128] of weight_dtype (fp32 or bf16), 4-byte (fp32) or
 * 2-byte (bf16) aligned; a null weight leaves that kind of row without a norm.
 * eps: finite, >= 0. */
typedef struct {
    const void *q_weight;
    const void *k_weight;
    nvfp4kv_dtype weight_dtype;
    float eps;
} nvfp4kv_head_norm;

/* q, k (no counterpart on the pages): num_tokens rows of [num_q_heads][128]
 *   and [num_kv_heads][128], fp32 or bf16 (in_dtype), token t's at q + t *
 *   q_stride (elements; at least the row, a multiple of 16 bytes, at most
 *   2^28), so parts of a fused projection's rows can be given as they are;
 *   16-byte aligned.
 * positions: int32 [num_tokens] (device); a token with a negative position is
 *   not there: its rows of the outputs are left as they are.
 * rope, norm: host structs, either may be NULL; their host data is read
 *   during the call.  Anything but the values above returns
 *   NVFP4KV_ERR_UNSUPPORTED.
 * q_out: bf16 [num_tokens][num_q_heads][128]; k_out: in_dtype
 *   [num_tokens][num_kv_heads][128]; 16-byte aligned.  q_out may be q and
 *   k_out may be k (same address, type and contiguous rows); any other overlap
 *   with an input returns NVFP4KV_ERR_INVALID_ARG. */
nvfp4kv_status nvfp4kv_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                    nvfp4kv_dtype in_dtype, int32_t num_tokens, int32_t num_q_heads,
                                    int32_t num_kv_heads, const int32_t *positions, const nvfp4kv_rope *rope,
                                    const nvfp4kv_head_norm *norm, void *q_out, void *k_out,
                                    int32_t *dev_status, nvfp4kv_stream_t stream);

/* The same fused with the cache write ("SGLang stores KV cache in 4 bits",
 * Interpretation: new K/V are quantised into the NVFP4 cache): q_out as above;
 * the finished keys, rounded to in_dtype, and the values v (rows as k's, at
 * v_stride) go into the cache at slot_mapping[t] exactly as
 * nvfp4kv_quantize_append would write them -- the keys are never stored
 * elsewhere.  num_kv_heads is the cache's.  slot < 0 or position < 0 writes
 * nothing of the token's K and V; slot >= num_pages * page_size likewise, and
 * sets NVFP4KV_DEV_BAD_SLOT.  Slots must be distinct. */
nvfp4kv_status nvfp4kv_qk_norm_rope_append(const nvfp4kv_cache *cache, const void *q, int64_t q_stride,
                                           const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                           nvfp4kv_dtype in_dtype, int32_t num_tokens, int32_t num_q_heads,
                                           const int32_t *positions, const int32_t *slot_mapping,
                                           const nvfp4kv_rope *rope, const nvfp4kv_head_norm *norm, void *q_out,
                                           int32_t *dev_status, nvfp4kv_stream_t stream);

/* FP8-E4M3 comparison cache, written and read the same way ("NVFP4-KV-Cache
 * auf der ...", "Unterstuetzung in den Engines": the FP8 baseline runs with
 * --kv-cache-dtype fp8_e4m3; "Bytes pro Token": scales 1.0 uncalibrated).
 * Each value is E4M3_rn_satfinite(x).  Arguments as for the NVFP4 calls. */
nvfp4kv_status fp8kv_quantize_append(const fp8kv_cache *cache, const void *k_new,
                                     const void *v_new, nvfp4kv_dtype in_dtype,
                                     int32_t num_tokens, const int32_t *slot_mapping,
                                     int32_t *dev_status, nvfp4kv_stream_t stream);

nvfp4kv_status fp8kv_paged_decode(const fp8kv_cache *cache, const void *q, int32_t batch,
                                  int32_t num_q_heads, const int32_t *block_table,
                                  int32_t max_pages_per_seq, const int32_t *seq_lens,
                                  float sm_scale, void *out, nvfp4kv_dtype out_dtype,
                                  void *workspace, size_t workspace_bytes,
                                  int32_t num_workers, int32_t *dev_status,
                                  nvfp4kv_stream_t stream);

/* The same fused step over the FP8 comparison cache (the FP8 baseline of
 * "NVFP4-KV-Cache auf der ...", "Unterstuetzung in den Engines", run through
 * the same append-then-decode step for a like-for-like comparison). */
nvfp4kv_status fp8kv_append_paged_decode(const fp8kv_cache *cache, const void *k_new, const void *v_new,
                                         nvfp4kv_dtype in_dtype, const void *q, int32_t batch,
                                         int32_t num_q_heads, const int32_t *block_table,
                                         int32_t max_pages_per_seq, const int32_t *seq_lens, float sm_scale,
                                         void *out, nvfp4kv_dtype out_dtype, void *workspace,
                                         size_t workspace_bytes, int32_t num_workers, int32_t *dev_status,
                                         nvfp4kv_stream_t stream);

/* ---- An FP8 cache with a scale for each page and kv head -----------------------
 *
 * The pages compare with an FP8 cache at scale 1.0 ("NVFP4-KV-Cache auf der
 * ...", "Bytes pro Token": uncalibrated), which saturates at 448 and loses small
 * values.  Here each page of a kv head has its own scale for K and for V (this
 * library's choice; the pages name calibration as the next step), found as
 * the tokens are written: with amax the largest magnitude of the block's new
 * values,
 *   s = 2^e, e the least integer with amax <= 448 * 2^e, from -100 to 100,
 *   code = E4M3_rn_satfinite(x / s)   (x / s is exact).
 * A page that holds tokens already keeps its scale unless new tokens need a
 * larger one; then the codes that are there are rounded anew,
 * E4M3_rn(code * s_old / s), which is exact but for codes that become subnormal.
 * A page whose first token comes with the call starts from that call's tokens.
 */

/* Write the last C = q_indptr[b+1] - q_indptr[b] tokens of sequence b's
 * seq_lens[b] tokens (a library utility: the write side of this cache; the
 * arguments are those of nvfp4kv_paged_extend, so that nvfp4kv_plan_step's
 * outputs fit).  Sequence b's rows are q_indptr[b] .. q_indptr[b+1] - 1 of
 *   k_new, v_new  [num_tokens][num_kv_heads][128], fp32 or bf16, 16-byte aligned
 * and go to positions seq_lens[b] - C .. seq_lens[b] - 1, in the pages that the
 * block table (int32 [batch][max_pages_per_seq]) lists.  Rows outside every
 * range are not read.  Positions of the last page behind the sequence hold
 * unspecified codes afterwards.  A page that receives tokens must not be in
 * another sequence's table.
 * A sequence whose range is outside [0, num_tokens], or whose length is less
 * than C or more than max_pages_per_seq * 16, is not written and sets
 * NVFP4KV_DEV_BAD_LEN; a page id outside [0, num_pages) is skipped and sets
 * NVFP4KV_DEV_BAD_PAGE.  q_indptr must not fall from one sequence to the next
 * (the rows behind one that does may be left out).  A call of no rows
 * (num_tokens 0) reads and sets nothing.  batch at most NVFP4KV_MAX_BATCH.
 * Non-finite inputs give unspecified codes. */
nvfp4kv_status fp8bkv_append(const fp8bkv_cache *cache, const void *k_new, const void *v_new, nvfp4kv_dtype in_dtype,
                             int32_t num_tokens, const int32_t *q_indptr, int32_t batch, const int32_t *block_table,
                             int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t *dev_status,
                             nvfp4kv_stream_t stream);

/* Read cached rows back (a library utility): for j < lens[b]
 *   k_out[kv_indptr[b] + j][h][c] = code * scale, rounded to out_dtype
 * (fp32 and bf16 hold it exactly, but for values past their range; NVFP4KV_E4M3
 * rounds and saturates: the FP8 workspace that the extend calls take, which has
 * no scales), v_out the same; each [rows][num_kv_heads][128], 16-byte aligned,
 * sized by the caller.  Cached values past 448, or so small that E4M3 at scale 1.0
 * has no bits for them, are not what that workspace holds: a prompt chunk that the
 * extend calls attend over it sees others there than the decodes, which apply the
 * scales.  Cached values of 0 or of magnitude 2^-6 .. 448 come
 * through as they are.
 * Lengths and page ids are checked as in nvfp4kv_paged_decode.  batch at most
 * NVFP4KV_MAX_BATCH.  k_out and v_out overlap neither one another nor anything
 * that is read; an output whose first row does is refused
 * (NVFP4KV_ERR_INVALID_ARG), the rows behind it are the device's to know. */
nvfp4kv_status fp8bkv_dequant(const fp8bkv_cache *cache, const int32_t *block_table, int32_t max_pages_per_seq,
                              const int32_t *lens, const int32_t *kv_indptr, int32_t batch, void *k_out, void *v_out,
                              nvfp4kv_dtype out_dtype, int32_t *dev_status, nvfp4kv_stream_t stream);

/* Decode attention over the block-scaled cache (a library utility with no
 * counterpart on the pages): q_len query tokens per sequence (1 ..
 * NVFP4KV_MAX_QUERY_TOKENS), causal among themselves, as in
 * nvfp4kv_paged_decode_multi.  Arguments, checks and results as there; seq_lens
 * and block_table are read ahead of the wait for the kernel before, too.  out and
 * the workspace overlap nothing else (NVFP4KV_ERR_INVALID_ARG).
 * Arithmetic: codes are exact in fp16, q too (bf16 significands under a power of
 * two a row; elements under 2^-28 of the row's largest lose bits); sm_scale and
 * a page's scales are applied in fp32, where scores, softmax and outputs are held;
 * softmax weights are rounded to fp16 for the value product, before the scale of
 * a page's values: a weight below 2^-25 of the row's largest counts as none, also
 * where its page's values are so much larger than the others'. */
nvfp4kv_status fp8bkv_paged_decode(const fp8bkv_cache *cache, const void *q, int32_t batch, int32_t q_len,
                                   int32_t num_q_heads, const int32_t *block_table, int32_t max_pages_per_seq,
                                   const int32_t *seq_lens, float sm_scale, void *out, nvfp4kv_dtype out_dtype,
                                   void *workspace, size_t workspace_bytes, int32_t num_workers, int32_t *dev_status,
                                   nvfp4kv_stream_t stream);

/* Bytes of a block-scaled FP8 pool; -1 for invalid arguments (a library utility;
 * host only).  Only the supported geometry has one. */
int64_t fp8bkv_cache_bytes(int32_t num_pages, int32_t num_kv_heads, int32_t page_size, int32_t head_dim);

/* ---- Attention over the pages that a query selects ------------------------------
 *
 * The pages read the whole cache at every step; these calls (with no counterpart
 * there) read, for each query token and kv head, the pages that a cheap score
 * puts first.  Three steps: bounds of the pages' keys, kept up as tokens are
 * written; the selection; decode over the selected pages.
 *
 * Bounds of a page and kv head over the page's cached tokens (values as cached,
 * without the tensor scale G): u = max |k|, r = fl32(127 / u),
 *   bounds[..][1][c] = min(127, ceil(fl32(max_t k[t][c] * r)))
 *   bounds[..][0][c] = max(-127, floor(fl32(min_t k[t][c] * r)))
 *   steps[..] = fl32(u / 127);   u = 0: all of them 0.
 */

/* Brings the bounds of sequence b's pages floor(from_lens[b] / 16) ..
 * ceil(seq_lens[b] / 16) - 1 up to date (a library utility): those that tokens
 * from_lens[b] .. seq_lens[b] - 1 were written into.  from_lens NULL: all pages.
 * After tokens were rejected the bounds of the last page are wider than need be
 * until it is written into again, never narrower.
 * A length outside [0, max_pages_per_seq * 16] is clamped and sets
 * NVFP4KV_DEV_BAD_LEN, as does a negative from_lens; a page id outside
 * [0, num_pages) is skipped and sets NVFP4KV_DEV_BAD_PAGE.  batch at most
 * NVFP4KV_MAX_BATCH.  bounds must have the cache's num_pages and
 * num_kv_heads (NVFP4KV_ERR_INVALID_ARG). */
nvfp4kv_status nvfp4kv_page_bounds(const nvfp4kv_cache *cache, const nvfp4kv_bounds *bounds,
                                   const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *from_lens,
                                   const int32_t *seq_lens, int32_t batch, int32_t *dev_status,
                                   nvfp4kv_stream_t stream);

/* The same of the block-scaled FP8 cache (a library utility). */
nvfp4kv_status fp8bkv_page_bounds(const fp8bkv_cache *cache, const nvfp4kv_bounds *bounds, const int32_t *block_table,
                                  int32_t max_pages_per_seq, const int32_t *from_lens, const int32_t *seq_lens,
                                  int32_t batch, int32_t *dev_status, nvfp4kv_stream_t stream);

/* Selects pages for each query token and kv head (a library utility, for either
 * cache).  Query token t of sequence b (q bf16 [batch][q_len][num_q_heads][128],
 * q_len 1 .. NVFP4KV_MAX_QUERY_TOKENS, the sequence's last positions) sees the
 * first n = seq_lens[b] - q_len + t + 1 tokens, so P = ceil(n / 16) pages (none
 * where n <= 0).  With the group's queries in whole steps, w = rint(fl32(q *
 * fl32(127 / max |q|))), the maximum over the group's heads and channels (where it
 * is below 2^-100, of queries 2^100 times as large, for the quotient's sake):
 *   score(page) = fl32(step * max_h sum_c max(w_hc * hi_c, w_hc * lo_c)),
 * the most that a key within the bounds can reach with one of the heads; the
 * sum is a whole number below 2^24, so the score depends on no order of sums.
 * A score past fp32's range counts as its largest finite number of that sign.
 * Selected are the first `first_pages` and the last `last_pages` of the P and the
 * others of the largest scores, the lower page where two are equal, `budget` in
 * all, or all P where they are no more than that.
 *   pages      int32 [batch][q_len][num_kv_heads][budget]: the selected pages'
 *              places in the sequence (indices into its row of the block table),
 *              ascending, -1 behind the last one
 * first_pages + last_pages at most budget; max_pages_per_seq at most
 * NVFP4KV_MAX_SELECT_PAGES (the scores stay in shared memory); batch * q_len at
 * most NVFP4KV_MAX_BATCH.  A length outside [0,
 * max_pages_per_seq * 16] is clamped and sets NVFP4KV_DEV_BAD_LEN; the score of a
 * page id outside [0, num_pages) is that of page 0 and sets
 * NVFP4KV_DEV_BAD_PAGE.  Non-finite queries give an unspecified selection (of
 * pages there are).  pages overlaps nothing else (NVFP4KV_ERR_INVALID_ARG).
 * seq_lens and block_table are read ahead of the wait for the kernel before, as
 * in nvfp4kv_paged_decode. */
#define NVFP4KV_MAX_SELECT_PAGES 65536
nvfp4kv_status nvfp4kv_select_pages(const nvfp4kv_bounds *bounds, const void *q, int32_t batch, int32_t q_len,
                                    int32_t num_q_heads, const int32_t *block_table, int32_t max_pages_per_seq,
                                    const int32_t *seq_lens, int32_t budget, int32_t first_pages, int32_t last_pages,
                                    int32_t *pages, int32_t *dev_status, nvfp4kv_stream_t stream);

/* Decode attention over listed pages (a library utility): query token t of
 * sequence b, kv head h attends over those of its first n = seq_lens[b] - q_len +
 * t + 1 tokens that lie in the first min(budget, ceil(n / 16)) entries of
 * pages[b][t][h] (as nvfp4kv_select_pages writes them; any order).  An entry
 * outside [0, ceil(n / 16)) has no tokens and sets NVFP4KV_DEV_BAD_PAGE; an entry
 * that is there twice counts twice.  A token that sees no key gets zeros.
 *   q    bf16 [batch][q_len][num_q_heads][128], out the same in out_dtype
 *   workspace, num_workers  as for nvfp4kv_paged_decode
 * batch * q_len at most NVFP4KV_MAX_BATCH; other arguments, checks and arithmetic
 * as for nvfp4kv_paged_decode, whose reading of seq_lens and block_table ahead of
 * the wait for the kernel before this call shares (pages is read behind it).  out
 * and the workspace overlap nothing else (NVFP4KV_ERR_INVALID_ARG). */
nvfp4kv_status nvfp4kv_selected_decode(const nvfp4kv_cache *cache, const void *q, int32_t batch, int32_t q_len,
                                       int32_t num_q_heads, const int32_t *block_table, int32_t max_pages_per_seq,
                                       const int32_t *seq_lens, const int32_t *pages, int32_t budget, float sm_scale,
                                       void *out, nvfp4kv_dtype out_dtype, void *workspace, size_t workspace_bytes,
                                       int32_t num_workers, int32_t *dev_status, nvfp4kv_stream_t stream);

/* The same over the block-scaled FP8 cache (a library utility), with
 * fp8bkv_paged_decode's arithmetic. */
nvfp4kv_status fp8bkv_selected_decode(const fp8bkv_cache *cache, const void *q, int32_t batch, int32_t q_len,
                                      int32_t num_q_heads, const int32_t *block_table, int32_t max_pages_per_seq,
                                      const int32_t *seq_lens, const int32_t *pages, int32_t budget, float sm_scale,
                                      void *out, nvfp4kv_dtype out_dtype, void *workspace, size_t workspace_bytes,
                                      int32_t num_workers, int32_t *dev_status, nvfp4kv_stream_t stream);

/* Bytes of an NVFP4 pool (K and V data and scales) for a geometry:
 * num_pages * num_kv_heads * page_size * 2 * (head_dim/2 + head_dim/16),
 * i.e. 9 bytes per 16 values ("SGLang stores KV cache in 4 bits",
 * Interpretation); for the supported geometry that is num_pages *
 * num_kv_heads * NVFP4KV_RECORD_BYTES.  Returns -1 for invalid arguments.
 * Host only. */
int64_t nvfp4kv_cache_bytes(int32_t num_pages, int32_t num_kv_heads, int32_t page_size,
                            int32_t head_dim);

/* Bytes of an FP8 pool: num_pages * num_kv_heads * page_size * 2 * head_dim,
 * one byte per value ("NVFP4-KV-Cache auf der ...", "Bytes pro Token: FP8
 * gegenueber NVFP4": 16 bytes per 16 values in FP8).  Returns -1 for invalid
 * arguments.  Host only. */
int64_t fp8kv_cache_bytes(int32_t num_pages, int32_t num_kv_heads, int32_t page_size,
                          int32_t head_dim);

/* A library utility with no counterpart on the pages: read a device status
 * word once the work on `stream` has finished:
 * synchronises the stream, copies *dev_status (device int32) into *bits
 * (host) and returns NVFP4KV_ERR_DEVICE_CHECK when any bit is set, NVFP4KV_OK
 * when none is (NVFP4KV_ERR_CUDA if the synchronisation or copy fails).  The
 * word is not reset.  Null pointers return NVFP4KV_ERR_INVALID_ARG. */
nvfp4kv_status nvfp4kv_read_device_status(const int32_t *dev_status, nvfp4kv_stream_t stream,
                                          int32_t *bits);

/* Failure detection (a library utility with no counterpart on the pages).
 * Every kernel wait for staged data, or for another part of the same CTA,
 * gives up after a number of polls, sets NVFP4KV_DEV_TIMEOUT in *dev_status,
 * lets whatever it already started (bulk copies, tensor-core operations)
 * finish and returns, so a wait that can never be satisfied costs a short
 * delay and a status bit, not a hung GPU.  This sets that number for the
 * calls made from now on in this process (0 = give up without polling;
 * NVFP4KV_WAIT_LIMIT_DEFAULT is the default) and returns the previous value.
 * The waits for work already in flight always use the default.  Host only,
 * thread-safe; a small limit makes ordinary calls report timeouts. */
#define NVFP4KV_WAIT_LIMIT_DEFAULT 4194304u
uint32_t nvfp4kv_set_wait_limit(uint32_t polls);

/* Static description of a status code (library utility). */
const char *nvfp4kv_status_string(nvfp4kv_status status);

/* Library version: major * 10000 + minor * 100 + patch (library utility). */
int32_t nvfp4kv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4KV_H */
