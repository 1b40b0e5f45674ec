// chunk_bf16_16.cu -- the chunk attention for bf16 queries over a cache of its own type.
#include "chunk_kernel.cuh"

namespace pkv {

cudaError_t chunk_bf16_16(const ChunkParams& p, int head_dim, cudaStream_t s) {
    return launch_chunk_kv<BF16, BF16>(p, head_dim, s);
}

}  // namespace pkv
