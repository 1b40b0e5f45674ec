// cache_ops.cuh -- parameters and host launchers of the cache-writing kernels.
#pragma once

#include "common.cuh"

namespace pkv {

// Launch a kernel that starts with pdl_launch_dependents() and pdl_wait(): its launch overlaps the
// end of the kernel before it on the stream (programmatic dependent launch), which hides 0.3 - 2 us
// of a call in a run of them (gather of one context 8.2 -> 5.8 us; the host's part is the same).
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned grid, unsigned threads,
                              cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

struct ReshapeParams {
    const void* key;
    const void* value;
    void* k_cache;
    void* v_cache;
    const int64_t* slot_mapping;
    unsigned* status;
    int num_tokens, num_kv_heads, head_dim, block_size, num_blocks;
    float kv_scale;
};

struct CopyParams {
    const void* src_k;    // source pool (device memory or mapped pinned host memory)
    const void* src_v;
    void* dst_k;          // destination pool (same pool for copy-on-write)
    void* dst_v;
    const int32_t* pairs;
    unsigned* status;
    int64_t block_bytes;   // num_kv_heads * block_size * bytes of a row
    int src_num_blocks, dst_num_blocks;
};

cudaError_t launch_reshape_and_cache(const ReshapeParams& p, pkv_dtype src, bool quant,
                                     int num_sms, cudaStream_t stream);
cudaError_t launch_reshape_and_cache_fp4(const ReshapeParams& p, pkv_dtype src, int num_sms,
                                         cudaStream_t stream);
cudaError_t launch_copy_blocks(const CopyParams& p, int num_pairs, cudaStream_t stream);

// Reading the cache back into contiguous rows (gather.cu).
struct GatherParams {
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* row_start;
    const int32_t* token_start;   // may be null: 0
    void* key_out;
    void* value_out;
    unsigned* status;
    int num_seqs, total_rows, num_kv_heads, head_dim, block_size, num_blocks, max_blocks;
    float kv_scale;
};

cudaError_t launch_gather_cache(const GatherParams& p, pkv_dtype kv, pkv_dtype out,
                                cudaStream_t stream);

// A kernel whose pipeline wait can never complete: it flags PKV_DEV_WAIT_TIMEOUT in
// `status` once the wait's bound has passed, and returns.
cudaError_t launch_wait_bound_probe(unsigned* status, cudaStream_t stream);

}  // namespace pkv
