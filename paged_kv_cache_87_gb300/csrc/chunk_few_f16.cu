// chunk_few_f16.cu -- the chunk attention of sequences with few rows, for f16 queries.
#include "chunk_few_kernel.cuh"

namespace pkv {

cudaError_t chunk_few_f16(const ChunkParams& p, int head_dim, pkv_dtype kv, cudaStream_t s) {
    return launch_chunk_few_q<F16>(p, head_dim, kv, s);
}

}  // namespace pkv
