// decode_fp4_f16.cu -- the decode over the 4-bit cache for f16 queries.
#include "decode_fp4_kernel.cuh"

namespace pkv {

cudaError_t decode_fp4_f16(const DecodeFp4Params& p, cudaStream_t s) { return launch_decode_fp4<F16>(p, s); }

}  // namespace pkv
