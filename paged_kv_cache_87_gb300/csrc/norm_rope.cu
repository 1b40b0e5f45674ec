// norm_rope.cu -- per-head RMS norm and rotary embedding of queries and keys in one pass,
// with or without the write of keys and values into the paged cache.
//
// For a head row x: y = x / sqrt(mean(x^2) + eps) * w, then every pair (y_i, y_j) of the first
// rot_dim dims is rotated by its angle.  One read and one write of every row: bound by HBM at
// prompt sizes, by the launch at a decode step's.
//
// A lane holds eight dims of a row (d / 8 lanes a row) as two runs of four: the halves of four
// pairs, so that the rotation stays in the lane (half-split: dims 4j .. and rot_dim / 2 + 4j ..;
// adjacent pairs and dims beyond rot_dim: eight in a row).  The sum of squares is a shuffle
// reduction over the row's lanes.  A warp takes kNormRows rows a lane group of one kind (query,
// key or value heads) of one token: weight times cosine and sine are formed once for them all,
// and their loads are in flight together.  Everything is fp32 until the one rounding at the end;
// with the cache write the keys are rounded to their own type first, so that the cache holds the
// same bits as after the two separate calls.
#include "norm_rope.cuh"

#include "cache_row.cuh"

namespace pkv {

constexpr int kNormThreads = 256;
constexpr int kNormRows = 4;     // rows a lane works on at once: their loads are in flight together

// What the kernel does with keys: NoCache writes k_out, a cache type writes the pool.
struct NoCache {};

// Four consecutive elements as stored (8 bytes of a 16-bit type, 16 of fp32) <-> fp32.
template <typename ST>
struct Four {
    using raw = typename std::conditional<ST::bytes == 4, uint4, uint2>::type;
    __device__ __forceinline__ static raw load(const void* p) { return *static_cast<const raw*>(p); }
    __device__ __forceinline__ static void to_float(const raw& r, float* f) {
        if constexpr (ST::bytes == 4) {
            Chunk<ST>::to_float(r, f);
        } else {
            float x[8];
            Chunk<ST>::to_float(make_uint4(r.x, r.y, 0u, 0u), x);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = x[i];
        }
    }
    __device__ __forceinline__ static raw pack(const float* f) {
        if constexpr (ST::bytes == 4) {
            return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                              __float_as_uint(f[3]));
        } else {
            const float x[8] = {f[0], f[1], f[2], f[3], 0.f, 0.f, 0.f, 0.f};
            const uint4 v = pack8<ST>(x);
            return make_uint2(v.x, v.y);
        }
    }
};

__device__ __forceinline__ uint2 shfl_raw(uint2 v, int src) {
    return make_uint2(__shfl_sync(0xffffffffu, v.x, src), __shfl_sync(0xffffffffu, v.y, src));
}
__device__ __forceinline__ uint4 shfl_raw(uint4 v, int src) {
    return make_uint4(__shfl_sync(0xffffffffu, v.x, src), __shfl_sync(0xffffffffu, v.y, src),
                      __shfl_sync(0xffffffffu, v.z, src), __shfl_sync(0xffffffffu, v.w, src));
}

template <typename ST>
__device__ __forceinline__ void load_weight4(const void* w, int f32, int at, float* f) {
    if (f32) Four<F32>::to_float(Four<F32>::load(static_cast<const float*>(w) + at), f);
    else Four<ST>::to_float(Four<ST>::load(static_cast<const uint8_t*>(w) + at * ST::bytes), f);
}

template <typename ST, typename KT, int HD>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_kernel(NormRopeParams p, int warps,
                                                                    int log_block) {
    pdl_launch_dependents();   // the attention launched next may start its launch now
    constexpr bool CACHE = !std::is_same<KT, NoCache>::value;
    constexpr int LPR = HD / 8, RPW = 32 / LPR, STEP = RPW * kNormRows;   // lanes a row, rows a warp
    using R = Four<ST>;
    const int lane = threadIdx.x & 31, j = lane % LPR, sub = lane / LPR;
    const int nq = (p.num_q_heads + STEP - 1) / STEP, nk = (p.num_kv_heads + STEP - 1) / STEP;
    const int pieces = nq + (CACHE ? 2 : 1) * nk;                // warps' work of a token
    const int tpc = max(1, (int)(blockDim.x / 32) / warps);      // tokens of the CTA
    const int64_t t = (int64_t)blockIdx.x * tpc + (threadIdx.x >> 5) / warps;
    if (t >= p.num_tokens) return;
    const int64_t pos = p.positions[t];
    int64_t slot = -1;
    if constexpr (CACHE) slot = p.slot_mapping[t];
    const bool cached = slot >= 0 && (slot >> log_block) < p.num_blocks;
    const int in_block = (int)(slot & ((1 << log_block) - 1));
    const int64_t tile_bytes = (int64_t)p.block_size * [] {
        if constexpr (CACHE) return cache_row_bytes_of<KT>(HD);
        else return 0;
    }();
    const int64_t tile0 = (slot >> log_block) * p.num_kv_heads;  // of kv head 0; used if cached
    // this lane's runs of four dims
    const int half = p.rot_dim / 2;
    const bool turned = 8 * j < p.rot_dim, split = turned && !p.interleaved;
    const int da = split ? 4 * j : 8 * j, db = split ? half + 4 * j : 8 * j + 4;

    for (int piece = (threadIdx.x >> 5) % warps; piece < pieces; piece += blockDim.x / 32) {
        const int kind = piece < nq ? 0 : piece < nq + nk ? 1 : 2;       // query, key, value
        const int heads = kind == 0 ? p.num_q_heads : p.num_kv_heads;
        const int h0 = (piece - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * STEP + sub;
        if constexpr (CACHE) {
            if (kind == 2) {                                     // values: moved as they are
                float x[kNormRows][8];
#pragma unroll
                for (int u = 0; u < kNormRows; ++u)
                    if (h0 + u * RPW < heads) {
                        load8<ST>(static_cast<const uint8_t*>(p.v) +
                                      (t * p.v_stride + (int64_t)(h0 + u * RPW) * HD + 8 * j) * ST::bytes, x[u]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
                    }
                if (!cached || pos < 0 || pos >= p.max_position) continue;
#pragma unroll
                for (int u = 0; u < kNormRows; ++u) {
                    const bool live = h0 + u * RPW < heads;
                    CacheRow<KT>::store(static_cast<uint8_t*>(p.v_cache) +
                                            (live ? (tile0 + h0 + u * RPW) * tile_bytes : 0),
                                        p.block_size, HD, in_block, j, x[u], p.kv_scale, live);
                }
                continue;
            }
        }
        const uint8_t* src = static_cast<const uint8_t*>(kind == 0 ? p.q : p.k) +
                             (t * (kind == 0 ? p.q_stride : p.k_stride) + (int64_t)h0 * HD) * ST::bytes;
        typename R::raw ra[kNormRows], rb[kNormRows];
#pragma unroll
        for (int u = 0; u < kNormRows; ++u) {
            ra[u] = rb[u] = typename R::raw{};
            if (h0 + u * RPW < heads) {
                ra[u] = R::load(src + (u * RPW * HD + da) * ST::bytes);
                rb[u] = R::load(src + (u * RPW * HD + db) * ST::bytes);
            }
        }
        const void* weight = kind == 0 ? p.q_weight : p.k_weight;
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f;
        if (weight != nullptr) {
            load_weight4<ST>(weight, p.weight_f32, da, w);
            load_weight4<ST>(weight, p.weight_f32, db, w + 4);
        }
        if (pos < 0 || pos >= p.max_position) {                  // the whole warp: one token
            if (piece == 0 && lane == 0) set_status(p.status, PKV_DEV_BAD_POSITION);
            return;
        }
        // every output is x_i m_i + x_partner n_i: m = weight cosine, n = -+ partner's weight sine.
        // Half-split lanes pair dim i of the first run with dim i of the second; the others hold
        // pairs (2i, 2i + 1).
        float m[8], n[8];
        const float* cs = p.cos_sin + pos * p.rot_dim;
        if (split) {
            float c[4], sn[4];
            Four<F32>::to_float(Four<F32>::load(cs + 4 * j), c);
            Four<F32>::to_float(Four<F32>::load(cs + half + 4 * j), sn);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[i] = w[i] * c[i];
                n[i] = -(w[i + 4] * sn[i]);
                m[i + 4] = w[i + 4] * c[i];
                n[i + 4] = w[i] * sn[i];
            }
        } else if (turned) {
            float c[4], sn[4];
            Four<F32>::to_float(Four<F32>::load(cs + 4 * j), c);
            Four<F32>::to_float(Four<F32>::load(cs + half + 4 * j), sn);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[2 * i] = w[2 * i] * c[i];
                n[2 * i] = -(w[2 * i + 1] * sn[i]);
                m[2 * i + 1] = w[2 * i + 1] * c[i];
                n[2 * i + 1] = w[2 * i] * sn[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = w[i];
        }
        uint8_t* dst = nullptr;
        if (kind == 0)
            dst = static_cast<uint8_t*>(p.q_out) + (t * p.q_out_stride + (int64_t)h0 * HD) * ST::bytes;
        else if constexpr (!CACHE)
            dst = static_cast<uint8_t*>(p.k_out) + (t * p.k_out_stride + (int64_t)h0 * HD) * ST::bytes;
#pragma unroll
        for (int u = 0; u < kNormRows; ++u) {
            const bool live = h0 + u * RPW < heads;
            float x[8], y[8];
            R::to_float(ra[u], x);
            R::to_float(rb[u], x + 4);
            float rs = 1.f;
            if (weight != nullptr) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int off = LPR / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                rs = rsqrtf(fmaf(ss, 1.f / HD, p.eps));
            }
            if (split) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], m[i], __fmul_rn(x[(i + 4) % 8], n[i])) * rs;
            } else if (turned) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], m[i], __fmul_rn(x[i ^ 1], n[i])) * rs;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = x[i] * m[i] * rs;
            }
            typename R::raw oa = R::pack(y), ob = R::pack(y + 4);
            if (!CACHE || kind == 0) {
                if (live) {
                    *reinterpret_cast<typename R::raw*>(dst + (u * RPW * HD + da) * ST::bytes) = oa;
                    *reinterpret_cast<typename R::raw*>(dst + (u * RPW * HD + db) * ST::bytes) = ob;
                }
            } else if constexpr (CACHE && !is_quantised<KT>()) {
                if (live && cached) {
                    uint8_t* to = static_cast<uint8_t*>(p.k_cache) + (tile0 + h0 + u * RPW) * tile_bytes +
                                  (int64_t)in_block * HD * ST::bytes;
                    *reinterpret_cast<typename R::raw*>(to + da * ST::bytes) = oa;
                    *reinterpret_cast<typename R::raw*>(to + db * ST::bytes) = ob;
                }
            } else if constexpr (CACHE) {
                // quantised caches take eight dims in a row, 8j ..: runs 2j and 2j + 1, which
                // half-split lanes hold as their first or second run
                if (!p.interleaved) {
                    typename R::raw run[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int dim = 8 * j + 4 * k;
                        const bool b = dim < p.rot_dim ? dim >= half : k == 1;
                        const int from = dim < half ? dim / 4 : dim < p.rot_dim ? (dim - half) / 4 : j;
                        const typename R::raw xa = shfl_raw(oa, sub * LPR + from);
                        const typename R::raw xb = shfl_raw(ob, sub * LPR + from);
                        run[k] = b ? xb : xa;
                    }
                    oa = run[0];
                    ob = run[1];
                }
                R::to_float(oa, y);
                R::to_float(ob, y + 4);
                CacheRow<KT>::store(static_cast<uint8_t*>(p.k_cache) +
                                        (live && cached ? (tile0 + h0 + u * RPW) * tile_bytes : 0),
                                    p.block_size, HD, in_block, j, y, p.kv_scale, live && cached);
            }
        }
        if constexpr (CACHE)
            if (piece == 0 && lane == 0 && slot >= 0 && !cached) set_status(p.status, PKV_DEV_BAD_SLOT);
    }
}

template <typename ST, typename KT>
cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
    constexpr bool CACHE = !std::is_same<KT, NoCache>::value;
    const int step = 256 / p.head_dim * kNormRows;            // rows of a warp
    const int need = (p.num_q_heads + step - 1) / step +
                     (CACHE ? 2 : 1) * ((p.num_kv_heads + step - 1) / step);   // warps of a token
    const int most = kNormThreads / 32, warps = need < most ? need : most, tpc = most / warps;
    const int log_block = p.block_size == 8 ? 3 : p.block_size == 16 ? 4 : 5;
    const unsigned grid = (unsigned)((p.num_tokens + tpc - 1) / tpc), threads = 32u * warps * tpc;
    if (p.head_dim == 128) qk_norm_rope_kernel<ST, KT, 128><<<grid, threads, 0, stream>>>(p, warps, log_block);
    else qk_norm_rope_kernel<ST, KT, 64><<<grid, threads, 0, stream>>>(p, warps, log_block);
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
