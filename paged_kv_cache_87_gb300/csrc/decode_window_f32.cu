// decode_window_f32.cu -- decode under a sliding window for fp32 queries (K/V in fp32 or FP8 e4m3).
#include "decode_launch.cuh"

namespace pkv {

cudaError_t decode_window_f32(const DecodeParams& p, pkv_dtype kv, int hpi, cudaStream_t s) {
    if (kv == PKV_FP8_E4M3)
        return p.head_dim == 128 ? dispatch_window<F32, E4M3, 128>(p, hpi, s) : dispatch_window<F32, E4M3, 64>(p, hpi, s);
    return p.head_dim == 128 ? dispatch_window<F32, F32, 128>(p, hpi, s) : dispatch_window<F32, F32, 64>(p, hpi, s);
}

}  // namespace pkv
