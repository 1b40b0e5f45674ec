// chunk_bf16_fp8.cu -- the chunk attention for bf16 queries over a cache of FP8.
#include "chunk_kernel.cuh"

namespace pkv {

cudaError_t chunk_bf16_fp8(const ChunkParams& p, int head_dim, cudaStream_t s) {
    return launch_chunk_kv<BF16, E4M3>(p, head_dim, s);
}

}  // namespace pkv
