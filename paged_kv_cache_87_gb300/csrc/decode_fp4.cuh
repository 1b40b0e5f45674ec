// decode_fp4.cuh -- parameters and host launcher of the decode over the 4-bit cache.
#pragma once

#include "common.cuh"

namespace pkv {

struct DecodeFp4Params {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    void* out;
    unsigned* status;
    int num_seqs, num_q_heads, num_kv_heads, group;
    int head_dim, block_size, num_blocks, max_blocks, max_context_len;
    float qk_scale_log2;   // scale * log2(e) * kv_scale
    float out_scale;       // kv_scale
};

cudaError_t launch_decode_fp4(const DecodeFp4Params& p, pkv_dtype q, cudaStream_t stream);

}  // namespace pkv
