// decode_fp4.cu -- single-query decode attention over the 4-bit paged cache.
//
// o = sum_t softmax_t(scale q.k_t) v_t with k, v = code * scale * kv_scale; kv_scale is folded
// into the logit scale and the output.  One CTA per (sequence, query head): its four warps take
// every fourth token, a lane d / 32 dims of it, with a running max and sum each, and merge at the
// end.
#include "decode_fp4.cuh"

#include "cache_row.cuh"

namespace pkv {

template <typename QT, int HD>
__global__ void __launch_bounds__(128) decode_fp4_kernel(DecodeFp4Params p) {
    constexpr int LPR = HD / 8, TPW = 32 / LPR, GROUPS = 4 * TPW;   // lanes a token, tokens a warp
    __shared__ float s_acc[GROUPS][HD], s_m[GROUPS], s_l[GROUPS];
    const int s = blockIdx.x / p.num_q_heads, qh = blockIdx.x % p.num_q_heads;
    const int kvh = qh / p.group, B = p.block_size;
    const int lane = threadIdx.x & 31, j = lane % LPR;
    const int grp = (threadIdx.x >> 5) * TPW + lane / LPR;
    const int cap = min(p.max_context_len, p.max_blocks * B);
    int ctx = p.context_lens[s];
    if (ctx < 0 || ctx > cap) {
        if (threadIdx.x == 0) set_status(p.status, PKV_DEV_BAD_CONTEXT);
        ctx = ctx < 0 ? 0 : cap;
    }
    float q[8], acc[8] = {0.f}, m = -INFINITY, l = 0.f;
    const int64_t row0 = ((int64_t)s * p.num_q_heads + qh) * HD;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = load_as_float<QT>(p.q, row0 + 8 * j + i) * p.qk_scale_log2;
    const int64_t tile_bytes = (int64_t)B * cache_row_bytes_of<E2M1>(HD);
    for (int t0 = 0; t0 < ctx; t0 += GROUPS) {
        const int t = t0 + grp;
        const bool live = t < ctx;
        float k[8] = {0.f}, v[8] = {0.f};
        if (live) {
            int blk = p.block_tables[(int64_t)s * p.max_blocks + t / B];
            if (blk < 0 || blk >= p.num_blocks) {
                set_status(p.status, PKV_DEV_BAD_BLOCK_ID);
                blk = 0;
            }
            const int64_t tile = ((int64_t)blk * p.num_kv_heads + kvh) * tile_bytes;
            CacheRow<E2M1>::load(static_cast<const uint8_t*>(p.k_cache) + tile, B, HD, t % B, j, k);
            CacheRow<E2M1>::load(static_cast<const uint8_t*>(p.v_cache) + tile, B, HD, t % B, j, v);
        }
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) z = fmaf(q[i], k[i], z);
#pragma unroll
        for (int off = LPR / 2; off >= 1; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
        if (live) {
            const float mn = fmaxf(m, z);
            const float r = exp2f(m - mn), e = exp2f(z - mn);
            l = l * r + e;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = acc[i] * r + e * v[i];
            m = mn;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s_acc[grp][8 * j + i] = acc[i];
    if (j == 0) {
        s_m[grp] = m;
        s_l[grp] = l;
    }
    __syncthreads();
    if (threadIdx.x < HD) {
        float M = -INFINITY, L = 0.f, A = 0.f;
        for (int g = 0; g < GROUPS; ++g) M = fmaxf(M, s_m[g]);
        for (int g = 0; g < GROUPS; ++g) {
            const float f = s_m[g] == -INFINITY ? 0.f : exp2f(s_m[g] - M);
            L = fmaf(s_l[g], f, L);
            A = fmaf(s_acc[g][threadIdx.x], f, A);
        }
        store_from_float<QT>(p.out, row0 + threadIdx.x, ctx > 0 ? A / L * p.out_scale : 0.f);
    }
}

template <typename QT>
cudaError_t launch(const DecodeFp4Params& p, cudaStream_t stream) {
    const unsigned grid = (unsigned)(p.num_seqs * p.num_q_heads);
    if (p.head_dim == 128) decode_fp4_kernel<QT, 128><<<grid, 128, 0, stream>>>(p);
    else decode_fp4_kernel<QT, 64><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_decode_fp4(const DecodeFp4Params& p, pkv_dtype q, cudaStream_t stream) {
    if (q == PKV_F32) return launch<F32>(p, stream);
    return q == PKV_F16 ? launch<F16>(p, stream) : launch<BF16>(p, stream);
}

}  // namespace pkv
