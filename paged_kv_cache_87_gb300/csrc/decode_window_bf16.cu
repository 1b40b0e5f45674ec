// decode_window_bf16.cu -- decode under a sliding window for bf16 queries (K/V in bf16, FP8 or 4 bits).
#include "decode_launch.cuh"
#include "decode_window_kernel.cuh"

namespace pkv {

cudaError_t window_kernel_bf16(const DecodeParams& p, pkv_dtype kv, cudaStream_t s) {
    if (kv == PKV_FP8_E4M3)
        return p.head_dim == 128 ? launch_decode_window<BF16, E4M3, 128>(p, s) : launch_decode_window<BF16, E4M3, 64>(p, s);
    if (kv == PKV_FP4_E2M1)
        return p.head_dim == 128 ? launch_decode_window<BF16, E2M1, 128>(p, s) : launch_decode_window<BF16, E2M1, 64>(p, s);
    return p.head_dim == 128 ? launch_decode_window<BF16, BF16, 128>(p, s) : launch_decode_window<BF16, BF16, 64>(p, s);
}

}  // namespace pkv
