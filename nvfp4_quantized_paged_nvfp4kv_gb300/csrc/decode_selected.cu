// Decode over listed pages, of either cache: instantiations and launchers of the worker
// split, which many rows of long lists take (312 rows of 256 pages in 4 bits: 42 us, by
// clusters 55) and every call that names its workers; decode_cluster.cu has the rest.
#include "decode_common.cuh"

namespace nvfp4kv {

template <class Fmt>
static cudaError_t launch_decode(const DecodeParams &p, cudaStream_t s)
{
    const size_t smem = decode_smem_bytes<Fmt, true>(p.batch);
    const cudaError_t e = allow_shared<decode_kernel<Fmt, false, true>>();
    if (e != cudaSuccess)
        return e;
    const int grid = (p.num_workers + kDecodeWarps - 1) / kDecodeWarps;
    return launch_pdl(decode_kernel<Fmt, false, true>, dim3(grid), dim3(kDecodeWarps * 32), smem, s, p);
}

cudaError_t launch_decode_selected_nvfp4(const DecodeParams &p, cudaStream_t s)
{
    return launch_decode<Nvfp4Format>(p, s);
}

cudaError_t launch_decode_selected_fp8_block(const DecodeParams &p, cudaStream_t s)
{
    return launch_decode<Fp8BlockFormat>(p, s);
}

} // namespace nvfp4kv
