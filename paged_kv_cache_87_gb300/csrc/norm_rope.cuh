// norm_rope.cuh -- parameters and host launcher of the norm + rotary kernel.
#pragma once

#include "common.cuh"

namespace pkv {

struct NormRopeParams {
    const void* q;
    const void* k;
    const void* v;            // null: no cache write
    const void* q_weight;     // null: no norm
    const void* k_weight;
    const float* cos_sin;
    const int64_t* positions;
    void* q_out;
    void* k_out;              // without the cache write
    void* k_cache;
    void* v_cache;
    const int64_t* slot_mapping;
    unsigned* status;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;   // elements
    int num_tokens, num_q_heads, num_kv_heads, head_dim;
    int max_position, rot_dim, interleaved;
    int weight_f32;           // weights in fp32 (else of the rows' type)
    int block_size, num_blocks;
    float eps, kv_scale;
};

cudaError_t launch_qk_norm_rope(const NormRopeParams& p, pkv_dtype dtype, cudaStream_t stream);
cudaError_t launch_qk_norm_rope_and_cache(const NormRopeParams& p, pkv_dtype dtype, pkv_dtype kv,
                                          cudaStream_t stream);

}  // namespace pkv
