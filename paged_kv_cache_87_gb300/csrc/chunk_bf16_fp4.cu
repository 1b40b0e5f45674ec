// chunk_bf16_fp4.cu -- the chunk attention for bf16 queries over a cache of 4 bits.
#include "chunk_kernel.cuh"

namespace pkv {

cudaError_t chunk_bf16_fp4(const ChunkParams& p, int head_dim, cudaStream_t s) {
    return launch_chunk_kv<BF16, E2M1>(p, head_dim, s);
}

}  // namespace pkv
