// Paged decode over the block-scaled FP8 cache: instantiations and launcher.
//
// Long sequences (decode_cluster.cu has the short ones): the worker split.  A page's
// scales cost four products of scores and one multiply-add a pair of outputs, in fp32,
// beside the matrix products.  Bound by HBM: six sequences of 128K to 160K with 48 + 8
// heads take 280 us for 1.81 GB, 0.95 of the copy rate.
#include "decode_common.cuh"

namespace nvfp4kv {

template <bool kMulti>
static cudaError_t launch_decode(const DecodeParams &p, cudaStream_t s)
{
    const size_t smem = decode_smem_bytes<Fp8BlockFormat>(p.batch);
    const cudaError_t e = allow_shared<decode_kernel<Fp8BlockFormat, kMulti>>();
    if (e != cudaSuccess)
        return e;
    const int grid = (p.num_workers + kDecodeWarps - 1) / kDecodeWarps;
    return launch_pdl(decode_kernel<Fp8BlockFormat, kMulti>, dim3(grid), dim3(kDecodeWarps * 32), smem, s, p);
}

cudaError_t launch_decode_fp8_block(const DecodeParams &p, cudaStream_t s)
{
    return p.q_len > 1 ? launch_decode<true>(p, s) : launch_decode<false>(p, s);
}

} // namespace nvfp4kv
