// decode_window_f16.cu -- decode under a sliding window for f16 queries (K/V in f16 or FP8 e4m3).
#include "decode_window_kernel.cuh"

namespace pkv {

cudaError_t decode_window_f16(const DecodeParams& p, pkv_dtype kv, int hpi, cudaStream_t s) {
    if (kv == PKV_FP8_E4M3) return dispatch_window_kv<F16, E4M3>(p, hpi, s);
    return dispatch_window_kv<F16, F16>(p, hpi, s);
}

}  // namespace pkv
