// decode_window_f32.cu -- decode under a sliding window for f32 queries (K/V in f32 or FP8 e4m3).
#include "decode_window_kernel.cuh"

namespace pkv {

cudaError_t decode_window_f32(const DecodeParams& p, pkv_dtype kv, int hpi, cudaStream_t s) {
    if (kv == PKV_FP8_E4M3) return dispatch_window_kv<F32, E4M3>(p, hpi, s);
    return dispatch_window_kv<F32, F32>(p, hpi, s);
}

}  // namespace pkv
