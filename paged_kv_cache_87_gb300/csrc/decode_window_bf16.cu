// decode_window_bf16.cu -- decode under a sliding window for bf16 queries (K/V in bf16 or FP8 e4m3).
#include "decode_window_kernel.cuh"

namespace pkv {

cudaError_t decode_window_bf16(const DecodeParams& p, pkv_dtype kv, int hpi, cudaStream_t s) {
    if (kv == PKV_FP8_E4M3) return dispatch_window_kv<BF16, E4M3>(p, hpi, s);
    return dispatch_window_kv<BF16, BF16>(p, hpi, s);
}

}  // namespace pkv
