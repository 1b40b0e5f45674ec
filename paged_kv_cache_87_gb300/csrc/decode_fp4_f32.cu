// decode_fp4_f32.cu -- the decode over the 4-bit cache for f32 queries.
#include "decode_fp4_kernel.cuh"

namespace pkv {

cudaError_t decode_fp4_f32(const DecodeFp4Params& p, cudaStream_t s) { return launch_decode_fp4<F32>(p, s); }

}  // namespace pkv
