// FP8-E4M3 paged decode (comparison kernel): instantiation and launcher.
#include "decode_common.cuh"

namespace nvfp4kv {

template <class Fmt>
static cudaError_t launch_decode(const DecodeParams &p, cudaStream_t s)
{
    const size_t smem = decode_smem_bytes<Fmt>(p.batch);
    const cudaError_t e = allow_shared<decode_kernel<Fmt, false>>();
    if (e != cudaSuccess)
        return e;
    const int grid = (p.num_workers + kDecodeWarps - 1) / kDecodeWarps;
    return launch_pdl(decode_kernel<Fmt, false>, dim3(grid), dim3(kDecodeWarps * 32), smem, s, p);
}

cudaError_t launch_decode_fp8(const DecodeParams &p, cudaStream_t s)
{
    return launch_decode<Fp8Format>(p, s);
}

} // namespace nvfp4kv
