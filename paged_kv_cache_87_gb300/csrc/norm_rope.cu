// norm_rope.cu -- per-head RMS norm and rotary embedding of queries and keys in one pass,
// with or without the write of keys and values into the paged cache.
//
// For a head row x: y = x / sqrt(mean(x^2) + eps) * w, then every pair (y_i, y_j) of the first
// rot_dim dims is rotated by its angle.  One read and one write of every row: bound by HBM at
// prompt sizes, by the launch at a decode step's.  Measured with the write into a cache of the rows'
// own type, bf16, 32 / 8 heads, d 128: 16,384 tokens 67 us (6.1 TB/s, 0.90 of the measured copy rate),
// 64 tokens 2.8 us; alone, f16, 40 / 40 heads, d 64, 3,001 tokens 12.7 us (0.72).
// Into a quantised cache the same takes 121 us in 4 bits (3.0 TB/s, 0.44) and 131 us in FP8 (0.43), 64
// tokens 3.9 and 4.2: the query pieces are no other work, so what is beyond 67 us is the key and value
// pieces', which a third of the warps do while the rest are through.  The two calls one after the other,
// whose write gives every warp such a piece, take 72 and 80 us (64 tokens 4.2 and 5.3; 1,000 tokens in
// 4 bits 9.5 against this call's 11.2).
//
// A lane holds eight dims of a row (d / 8 lanes a row) as two runs of four: the halves of four
// pairs, so that the rotation stays in the lane (half-split: dims 4j .. and rot_dim / 2 + 4j ..;
// adjacent pairs and dims beyond rot_dim: eight in a row).  The sum of squares is a shuffle
// reduction over the row's lanes.  A warp takes kNormRows rows a lane group of one kind (query,
// key or value heads) of one token: weight times cosine and sine are formed once for them all,
// and their loads are in flight together.  The grid is what the device holds at once, and a warp
// walks the tokens with the next one's rows loading (a CTA a token took 101 us on the prompts).
// Everything is fp32 until the one rounding at the end;
// with the cache write the keys are rounded to their own type first, so that the cache holds the
// same bits as after the two separate calls.
#include "norm_rope.cuh"

#include "cache_ops.cuh"
#include "cache_row.cuh"

namespace pkv {

constexpr int kNormThreads = 128;   // (256: 68.5 us on the prompts against 67.2, one token 2.5 against 2.3)
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

// What a warp has loaded of one token: its rows as stored, their angles, the token's position and
// slot.
template <typename ST>
struct TokenRows {
    typename Four<ST>::raw a[kNormRows], b[kNormRows];
    float4 c, s;
    int64_t pos, slot;
};

template <typename ST, typename KT, int HD>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_kernel(NormRopeParams p, int log_block) {
    pdl_launch_dependents();   // the attention launched next may start its launch now
    pdl_wait();
    constexpr bool CACHE = !std::is_same<KT, NoCache>::value;
    constexpr int LPR = HD / 8, RPW = 32 / LPR, STEP = RPW * kNormRows;   // lanes a row, rows a warp
    using R = Four<ST>;
    const int lane = threadIdx.x & 31, j = lane % LPR, sub = lane / LPR;
    const int nq = (p.num_q_heads + STEP - 1) / STEP, nk = (p.num_kv_heads + STEP - 1) / STEP;
    const int pieces = nq + (CACHE ? 2 : 1) * nk;                // warps' work of a token
    const int gw = blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
    const int step = gridDim.x * (kNormThreads / 32) / pieces;   // tokens at work at once
    int64_t t = gw / pieces;
    if (t >= step || t >= p.num_tokens) return;
    const int piece = gw % pieces;
    const int kind = piece < nq ? 0 : piece < nq + nk ? 1 : 2;   // query, key, value heads
    const int heads = kind == 0 ? p.num_q_heads : p.num_kv_heads;
    const int h0 = (piece - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * STEP + sub;
    const int tile_bytes = p.block_size * [] {
        if constexpr (CACHE) return cache_row_bytes_of<KT>(HD);
        else return 0;
    }();
    // the tile of this lane's first row in the slot's block, and whether there is one
    auto tile_of = [&](int64_t slot) {
        return ((slot >> log_block) * p.num_kv_heads + h0) * (int64_t)tile_bytes;
    };
    auto cached = [&](int64_t slot) { return slot >= 0 && (slot >> log_block) < p.num_blocks; };
    auto known = [&](int64_t pos) { return pos >= 0 && pos < p.max_position; };

    if constexpr (CACHE) {
        if (kind == 2) {                                         // values: moved as they are
            uint4 x[kNormRows][ST::bytes / 2];
            auto fetch = [&](int64_t at) {
                const uint8_t* src = static_cast<const uint8_t*>(p.v) +
                                     (at * p.v_stride + h0 * HD + 8 * j) * ST::bytes;
#pragma unroll
                for (int u = 0; u < kNormRows; ++u)
#pragma unroll
                    for (int i = 0; i < ST::bytes / 2; ++i)
                        x[u][i] = h0 + u * RPW < heads
                            ? reinterpret_cast<const uint4*>(src + u * RPW * HD * ST::bytes)[i]
                            : make_uint4(0u, 0u, 0u, 0u);
            };
            for (; t < p.num_tokens; t += step) {
                fetch(t);
                const int64_t pos = p.positions[t], slot = p.slot_mapping[t];
                if (!cached(slot) || !known(pos)) continue;
                const int row = (int)(slot & ((1 << log_block) - 1));
                uint8_t* tile = static_cast<uint8_t*>(p.v_cache) + tile_of(slot);
#pragma unroll
                for (int u = 0; u < kNormRows; ++u) {
                    const bool live = h0 + u * RPW < heads;
                    uint8_t* to = tile + u * RPW * tile_bytes;
                    if constexpr (is_quantised<KT>()) {
                        float f[8];
                        load8<ST>(x[u], f);
                        CacheRow<KT>::store(to, p.block_size, HD, row, j, f, p.kv_scale, live);
                    } else if (live) {
                        CacheRow<KT>::put(to, HD, row, j, x[u]);
                    }
                }
            }
            return;
        }
    }

    // this lane's runs of four dims, and its weights
    const int half = p.rot_dim / 2;
    const bool turned = 8 * j < p.rot_dim, split = turned && !p.interleaved;
    const int da = split ? 4 * j : 8 * j, db = split ? half + 4 * j : 8 * j + 4;
    const void* weight = kind == 0 ? p.q_weight : p.k_weight;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (weight != nullptr) {
        load_weight4<ST>(weight, p.weight_f32, da, w);
        load_weight4<ST>(weight, p.weight_f32, db, w + 4);
    }
    const int64_t stride = kind == 0 ? p.q_stride : p.k_stride;
    const uint8_t* src = static_cast<const uint8_t*>(kind == 0 ? p.q : p.k) + (int64_t)h0 * HD * ST::bytes;
    int64_t out_stride = p.q_out_stride;
    uint8_t* out = static_cast<uint8_t*>(p.q_out) + (int64_t)h0 * HD * ST::bytes;
    if constexpr (!CACHE)
        if (kind == 1) {
            out_stride = p.k_out_stride;
            out = static_cast<uint8_t*>(p.k_out) + (int64_t)h0 * HD * ST::bytes;
        }
    auto fetch_rows = [&](TokenRows<ST>& r, int64_t at) {
        const uint8_t* row = src + at * stride * ST::bytes;
#pragma unroll
        for (int u = 0; u < kNormRows; ++u) {
            r.a[u] = r.b[u] = typename R::raw{};
            if (h0 + u * RPW < heads) {
                r.a[u] = R::load(row + (u * RPW * HD + da) * ST::bytes);
                r.b[u] = R::load(row + (u * RPW * HD + db) * ST::bytes);
            }
        }
        r.slot = -1;
        if constexpr (CACHE) r.slot = p.slot_mapping[at];
    };
    auto fetch_angles = [&](TokenRows<ST>& r) {
        r.c = r.s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (turned && known(r.pos)) {
            const float* cs = p.cos_sin + r.pos * p.rot_dim + 4 * j;
            r.c = *reinterpret_cast<const float4*>(cs);
            r.s = *reinterpret_cast<const float4*>(cs + half);
        }
    };

    // rows and angles load one token ahead, positions two
    TokenRows<ST> now, next;
    now.pos = p.positions[t];
    int64_t pos_after = t + step < p.num_tokens ? p.positions[t + step] : 0;
    fetch_rows(now, t);
    fetch_angles(now);
    for (; t < p.num_tokens; t += step) {
        if (t + step < p.num_tokens) {
            next.pos = pos_after;
            fetch_rows(next, t + step);
            fetch_angles(next);
            if (t + 2 * step < p.num_tokens) pos_after = p.positions[t + 2 * step];
        }
        if (!known(now.pos)) {                                   // the whole warp: one token
            if (piece == 0 && lane == 0) set_status(p.status, PKV_DEV_BAD_POSITION);
            now = next;
            continue;
        }
        // every output is x_i m_i + x_partner n_i: m = weight cosine, n = -+ partner's weight sine.
        // Half-split lanes pair dim i of the first run with dim i of the second; the others hold
        // pairs (2i, 2i + 1).
        float m[8], n[8];
        const float c[4] = {now.c.x, now.c.y, now.c.z, now.c.w};
        const float sn[4] = {now.s.x, now.s.y, now.s.z, now.s.w};
        if (split) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[i] = w[i] * c[i];
                n[i] = -(w[i + 4] * sn[i]);
                m[i + 4] = w[i + 4] * c[i];
                n[i + 4] = w[i] * sn[i];
            }
        } else if (turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[2 * i] = w[2 * i] * c[i];
                n[2 * i] = -(w[2 * i + 1] * sn[i]);
                m[2 * i + 1] = w[2 * i + 1] * c[i];
                n[2 * i + 1] = w[2 * i] * sn[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[i] = w[i];
                n[i] = 0.f;
            }
        }
        const bool hit = cached(now.slot);
        const int in_block = (int)(now.slot & ((1 << log_block) - 1));
        uint8_t* dst = out + t * out_stride * ST::bytes;
        uint8_t* tile = nullptr;
        if constexpr (CACHE)
            if (hit) tile = static_cast<uint8_t*>(p.k_cache) + tile_of(now.slot);
#pragma unroll
        for (int u = 0; u < kNormRows; ++u) {
            const bool live = h0 + u * RPW < heads;
            float x[8], y[8];
            R::to_float(now.a[u], x);
            R::to_float(now.b[u], x + 4);
            float rs = 1.f;
            if (weight != nullptr) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int off = LPR / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                rs = rsqrtf(fmaf(ss, 1.f / HD, p.eps));
            }
            // (a dim that is not rotated has n = 0, and its partner must not reach it as NaN)
            if (!p.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(turned ? x[(i + 4) % 8] : 0.f, n[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(turned ? x[i ^ 1] : 0.f, n[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], m[i], y[i]) * rs;
            typename R::raw oa = R::pack(y), ob = R::pack(y + 4);
            if (!CACHE || kind == 0) {
                if (live) {
                    *reinterpret_cast<typename R::raw*>(dst + (u * RPW * HD + da) * ST::bytes) = oa;
                    *reinterpret_cast<typename R::raw*>(dst + (u * RPW * HD + db) * ST::bytes) = ob;
                }
            } else if constexpr (CACHE && !is_quantised<KT>()) {
                if (live && hit) {
                    uint8_t* to = tile + u * RPW * tile_bytes + in_block * HD * ST::bytes;
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
                CacheRow<KT>::store(tile + (hit ? u * RPW * tile_bytes : 0), p.block_size, HD,
                                    in_block, j, y, p.kv_scale, live && hit);
            }
        }
        if constexpr (CACHE)
            if (piece == 0 && lane == 0 && now.slot >= 0 && !hit) set_status(p.status, PKV_DEV_BAD_SLOT);
        now = next;
    }
}

template <typename ST, typename KT, int HD>
cudaError_t launch_norm_rope_d(const NormRopeParams& p, cudaStream_t stream) {
    constexpr bool CACHE = !std::is_same<KT, NoCache>::value;
    constexpr int STEP = 256 / HD * kNormRows, WARPS = kNormThreads / 32;
    static int resident[64] = {0};                // CTAs the device holds at once
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    auto kernel = qk_norm_rope_kernel<ST, KT, HD>;
    if (resident[dev] == 0) {
        int per_sm = 0, sms = 0;
        err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kNormThreads, 0);
        if (err != cudaSuccess) return err;
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (err != cudaSuccess) return err;
        resident[dev] = (per_sm > 0 ? per_sm : 1) * sms;
    }
    const int64_t pieces = (p.num_q_heads + STEP - 1) / STEP +
                           (CACHE ? 2 : 1) * ((p.num_kv_heads + STEP - 1) / STEP);
    const int64_t least = (pieces + WARPS - 1) / WARPS;          // one token at work at least
    const int64_t most = resident[dev] > least ? resident[dev] : least;
    const int64_t need = (p.num_tokens * pieces + WARPS - 1) / WARPS;
    const int log_block = p.block_size == 8 ? 3 : p.block_size == 16 ? 4 : 5;
    return launch_overlapped(kernel, (unsigned)(need < most ? need : most), kNormThreads, stream, p,
                             log_block);
}

template <typename ST, typename KT>
cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
    return p.head_dim == 128 ? launch_norm_rope_d<ST, KT, 128>(p, stream)
                             : launch_norm_rope_d<ST, KT, 64>(p, stream);
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
