// chunk_f16_16.cu -- the chunk attention for f16 queries over a cache of its own type.
#include "chunk_kernel.cuh"

namespace pkv {

cudaError_t chunk_f16_16(const ChunkParams& p, int head_dim, cudaStream_t s) {
    return launch_chunk_kv<F16, F16>(p, head_dim, s);
}

}  // namespace pkv
