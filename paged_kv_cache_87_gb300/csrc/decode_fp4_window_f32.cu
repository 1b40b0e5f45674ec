// decode_fp4_window_f32.cu -- the decode over the 4-bit cache under a sliding window, f32 queries.
#include "decode_fp4_kernel.cuh"

namespace pkv {

cudaError_t decode_fp4_window_f32(const DecodeFp4Params& p, cudaStream_t s) {
    return launch_decode_fp4<F32, true>(p, s);
}

}  // namespace pkv
