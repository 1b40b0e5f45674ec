// decode_fp4_bf16.cu -- the decode over the 4-bit cache for bf16 queries.
#include "decode_fp4_kernel.cuh"

namespace pkv {

cudaError_t decode_fp4_bf16(const DecodeFp4Params& p, cudaStream_t s) { return launch_decode_fp4<BF16>(p, s); }

}  // namespace pkv
