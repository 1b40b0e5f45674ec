// norm_rope.cu -- per-head RMS norm and rotary embedding of queries and keys in one pass,
// with or without the write of keys and values into the paged cache.
//
// For a head row x: y = x / sqrt(mean(x^2) + eps) * w, then every pair (y_i, y_j) of the first
// rot_dim dims is rotated by its angle.  One read and one write of every row: bound by HBM at
// prompt sizes, by the launch at a decode step's.
//
// A lane holds eight consecutive dims of a row (d / 8 lanes a row, 32 * 8 / d rows a warp).  The
// sum of squares is a shuffle reduction over the row's lanes.  Half-split pairs lie rot_dim / 16
// lanes apart (eight shuffles; rot_dim is a multiple of 16, so a lane's eight dims are all in one
// half); adjacent pairs lie in the lane.  Everything is fp32 until the one rounding at the end;
// with the cache write the keys are rounded to their own type first, so that the cache holds the
// same bits as after the two separate calls.
#include "norm_rope.cuh"

#include "cache_row.cuh"

namespace pkv {

constexpr int kNormThreads = 256;

// What the kernel does with keys: NoCache writes k_out, a cache type writes the pool.
struct NoCache {};

template <typename ST>
__device__ __forceinline__ void load_weight8(const void* w, int f32, int j, float (&f)[8]) {
    if (f32) load8<F32>(static_cast<const float*>(w) + 8 * j, f);
    else load8<ST>(static_cast<const uint8_t*>(w) + (int64_t)8 * j * ST::bytes, f);
}

template <typename ST, typename KT, int HD>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_kernel(NormRopeParams p) {
    pdl_launch_dependents();   // the attention launched next may start its launch now
    constexpr bool CACHE = !std::is_same<KT, NoCache>::value;
    constexpr int LPR = HD / 8, RPW = 32 / LPR;       // lanes a row, rows a warp
    const int lane = threadIdx.x & 31, j = lane % LPR;
    const int rows = p.num_q_heads + (CACHE ? 2 : 1) * p.num_kv_heads;   // of a token
    const int per_token = (rows + RPW - 1) / RPW;                        // warps of a token
    const int64_t gw = (int64_t)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = gw / per_token;
    if (t >= p.num_tokens) return;
    const int r = (int)(gw % per_token) * RPW + lane / LPR;   // q heads, k heads, then v heads
    const int64_t pos = p.positions[t];
    if (pos < 0 || pos >= p.max_position) {
        if (r == 0 && j == 0) set_status(p.status, PKV_DEV_BAD_POSITION);
        return;                                               // the whole warp: one token
    }
    const bool in = r < rows;
    const bool is_q = r < p.num_q_heads;
    const bool is_v = CACHE && r >= p.num_q_heads + p.num_kv_heads;
    const int h = is_q ? r : (r - p.num_q_heads) % p.num_kv_heads;
    float x[8] = {0.f};
    if (in) {
        const void* base = is_q ? p.q : is_v ? p.v : p.k;
        const int64_t stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
        load8<ST>(static_cast<const uint8_t*>(base) +
                      (t * stride + (int64_t)h * HD + 8 * j) * ST::bytes, x);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const void* weight = is_q ? p.q_weight : p.k_weight;
    if (in && !is_v && weight != nullptr) {
        const float rs = __frsqrt_rn(ss * (1.f / HD) + p.eps);
        float w[8];
        load_weight8<ST>(weight, p.weight_f32, j, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * rs * w[i];
    }
    // rotation: lanes of v rows and of dims beyond rot_dim keep x
    const int half = p.rot_dim / 2;
    const float* cs = p.cos_sin + pos * p.rot_dim;
    const bool turned = in && !is_v && 8 * j < p.rot_dim;
    if (p.interleaved) {
        if (turned) {
            const float4 c = *reinterpret_cast<const float4*>(cs + 4 * j);
            const float4 s = *reinterpret_cast<const float4*>(cs + half + 4 * j);
            const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = a * cc[i] - b * sn[i];
                x[2 * i + 1] = b * cc[i] + a * sn[i];
            }
        }
    } else {
        const int dist = p.rot_dim / 16;              // lanes between the halves of a pair
        const bool low = 8 * j < half;
        const int src = turned ? (low ? lane + dist : lane - dist) : lane;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], src);
        if (turned) {
            const int f0 = low ? 8 * j : 8 * j - half;
            float c[8], s[8];
            load8<F32>(cs + f0, c);
            load8<F32>(cs + half + f0, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * c[i] + (low ? -y[i] : y[i]) * s[i];
        }
    }
    if (in && is_q)
        store8<ST>(static_cast<uint8_t*>(p.q_out) +
                       (t * p.q_out_stride + (int64_t)h * HD + 8 * j) * ST::bytes, x);
    if constexpr (!CACHE) {
        if (in && !is_q)
            store8<ST>(static_cast<uint8_t*>(p.k_out) +
                           (t * p.k_out_stride + (int64_t)h * HD + 8 * j) * ST::bytes, x);
    } else {
        const int64_t slot = p.slot_mapping[t];
        const bool inside = slot < (int64_t)p.num_blocks * p.block_size;
        if (!inside && r == 0 && j == 0) set_status(p.status, PKV_DEV_BAD_SLOT);
        const bool live = in && !is_q && slot >= 0 && inside;
        if constexpr (ST::bytes == 2) {               // the key in its own type first
            const uint4 raw = pack8<ST>(x);
            Chunk<ST>::to_float(raw, x);
        }
        const int64_t blk = live ? slot / p.block_size : 0;
        const int row = live ? (int)(slot % p.block_size) : 0;
        const int64_t tile = (blk * p.num_kv_heads + h) * p.block_size *
                             (int64_t)cache_row_bytes_of<KT>(HD);
        CacheRow<KT>::store(static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + tile,
                            p.block_size, HD, row, j, x, p.kv_scale, live);
    }
}

template <typename ST, typename KT>
cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
    constexpr bool CACHE = !std::is_same<KT, NoCache>::value;
    const int rpw = 256 / p.head_dim;
    const int rows = p.num_q_heads + (CACHE ? 2 : 1) * p.num_kv_heads;
    const int64_t warps = (int64_t)p.num_tokens * ((rows + rpw - 1) / rpw);
    const int64_t grid = (warps + kNormThreads / 32 - 1) / (kNormThreads / 32);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.head_dim == 128)
        qk_norm_rope_kernel<ST, KT, 128><<<(unsigned)grid, kNormThreads, 0, stream>>>(p);
    else
        qk_norm_rope_kernel<ST, KT, 64><<<(unsigned)grid, kNormThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const NormRopeParams& p, pkv_dtype dtype, cudaStream_t stream) {
    if (dtype == PKV_F32) return launch_norm_rope<F32, NoCache>(p, stream);
    return dtype == PKV_F16 ? launch_norm_rope<F16, NoCache>(p, stream)
                            : launch_norm_rope<BF16, NoCache>(p, stream);
}

template <typename ST>
cudaError_t dispatch_cache(const NormRopeParams& p, pkv_dtype kv, cudaStream_t stream) {
    if (kv == PKV_FP4_E2M1) return launch_norm_rope<ST, E2M1>(p, stream);
    if (kv == PKV_FP8_E4M3) return launch_norm_rope<ST, E4M3>(p, stream);
    return launch_norm_rope<ST, ST>(p, stream);
}

cudaError_t launch_qk_norm_rope_and_cache(const NormRopeParams& p, pkv_dtype dtype, pkv_dtype kv,
                                          cudaStream_t stream) {
    if (dtype == PKV_F32) return dispatch_cache<F32>(p, kv, stream);
    return dtype == PKV_F16 ? dispatch_cache<F16>(p, kv, stream)
                            : dispatch_cache<BF16>(p, kv, stream);
}

}  // namespace pkv
