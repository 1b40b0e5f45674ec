// cache_ops.cu -- the kernels that write the paged KV cache.
//
//  * reshape_and_cache ("PagedAttention: Mathematical Foundations ..." §7
//    kernel 1, "Fused Reshape and Block Write"): each new token's key and
//    value rows go straight to their physical slot, optionally quantised to
//    FP8 e4m3 with a per-tensor scale.
//  * copy_blocks (§5 Parallel Sampling step 4 and §7 kernel 3, "Batched Block
//    Copy-on-Write"): every copy-on-write block copy of a step in one launch.
//  * swap_blocks (§6 Preemption, swapping): the same batched block copy
//    between two pools, one of which may be pinned host memory that the GPU
//    reaches directly (NVLink-C2C on Grace-based systems).
// All are pure data movement: one thread moves one 16-byte chunk per
// iteration with vector loads/stores, in a grid-stride loop.
#include "cache_ops.cuh"
#include "cache_row.cuh"

namespace pkv {

template <typename ST>
__device__ __forceinline__ void load16_as_float(const uint8_t* src, float* f);

template <>
__device__ __forceinline__ void load16_as_float<F32>(const uint8_t* src, float* f) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
#pragma unroll
    for (int i = 0; i < 4; ++i) Chunk<F32>::to_float(s[i], f + 4 * i);
}
template <>
__device__ __forceinline__ void load16_as_float<F16>(const uint8_t* src, float* f) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
#pragma unroll
    for (int i = 0; i < 2; ++i) Chunk<F16>::to_float(s[i], f + 8 * i);
}
template <>
__device__ __forceinline__ void load16_as_float<BF16>(const uint8_t* src, float* f) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
#pragma unroll
    for (int i = 0; i < 2; ++i) Chunk<BF16>::to_float(s[i], f + 8 * i);
}

// One thread = one 16-byte chunk of one (token, kv head) row of the cache.
template <typename ST, bool QUANT>
__global__ void __launch_bounds__(256) reshape_and_cache_kernel(ReshapeParams p) {
    pdl_launch_dependents();   // the decode launched next may start its launch now
    constexpr int KB = QUANT ? 1 : ST::bytes;          // cache element bytes
    const int row_chunks = p.head_dim * KB / 16;
    const int64_t total = (int64_t)p.num_tokens * p.num_kv_heads * row_chunks;
    const int64_t pool_slots = (int64_t)p.num_blocks * p.block_size;
    for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < total;
         idx += (int64_t)gridDim.x * blockDim.x) {
        const int c = (int)(idx % row_chunks);
        const int64_t th = idx / row_chunks;
        const int h = (int)(th % p.num_kv_heads);
        const int64_t t = th / p.num_kv_heads;
        const int64_t slot = p.slot_mapping[t];
        if (slot < 0) continue;
        if (slot >= pool_slots) {
            if (c == 0 && h == 0) set_status(p.status, PKV_DEV_BAD_SLOT);
            continue;
        }
        const int64_t blk = slot / p.block_size, off = slot % p.block_size;
        const int64_t drow = ((blk * p.num_kv_heads + h) * p.block_size + off) * p.head_dim;
        const int64_t srow = (t * p.num_kv_heads + h) * p.head_dim;
        if constexpr (!QUANT) {
            const int64_t db = drow * KB + (int64_t)c * 16, sb = srow * KB + (int64_t)c * 16;
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.k_cache) + db) =
                *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.key) + sb);
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.v_cache) + db) =
                *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.value) + sb);
        } else {
            // 16 cache elements from 16 source elements
            const int64_t e0 = (int64_t)c * 16;
            const int64_t sb = (srow + e0) * ST::bytes;
            const void* srcs[2] = {p.key, p.value};
            void* dsts[2] = {p.k_cache, p.v_cache};
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                float f[16];
                load16_as_float<ST>(static_cast<const uint8_t*>(srcs[kv]) + sb, f);
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = __fdiv_rn(f[4 * i + 0], p.kv_scale);
                    const float b = __fdiv_rn(f[4 * i + 1], p.kv_scale);
                    const float cc = __fdiv_rn(f[4 * i + 2], p.kv_scale);
                    const float d = __fdiv_rn(f[4 * i + 3], p.kv_scale);
                    w[i] = cvt_e4m3x2(a, b) | (cvt_e4m3x2(cc, d) << 16);
                }
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(dsts[kv]) + drow + e0) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// Into the 4-bit cache.  A lane holds 16 dims of a (token, kv head) row: one scale's group, so that
// what a scale costs (a division, a reciprocal) is paid once.  A warp keeps its piece of a token --
// kWriteRows rows a lane group of K or of V -- and walks the tokens with the next token's rows and
// slot loading while it quantises this one's.  Bound by the arithmetic (173 instructions for a lane's
// 16 elements, 64 % of the issue slots): 32,768 tokens of 8 heads, d 128, bf16 in 34 us (5.1 TB/s) where
// HBM alone would take 25, with slots that fill block by block; in no order at all, 53 us.  (A lane of
// eight dims and an IEEE division each took 70 us.)
constexpr int kWriteRows = 2;
constexpr int kWriteThreads = 256;
// A SM's share of the grid: twice what is resident (three CTAs at 77 registers; two of fp32 rows, at
// 100).  Measured, 8 heads of 128: 32,768 tokens in bf16 34.0 us against 36.6 with three a SM, in fp32
// 49.7 against 51.3 with two; smaller chunks are better off with three (9,000 tokens 9.6 us against 10.4,
// 2,000 tokens 4.2 against 4.7), heads of 64 nearly the same (19.2 against 19.7).
constexpr int kWriteCtas = 6;

template <typename ST, int HD>
__global__ void __launch_bounds__(kWriteThreads) reshape_and_cache_fp4_kernel(ReshapeParams p,
                                                                              int log_block) {
    pdl_launch_dependents();   // the decode launched next may start its launch now
    pdl_wait();
    constexpr int LPR = HD / 16, RPW = 32 / LPR, STEP = RPW * kWriteRows;
    constexpr int TILE_ROW = cache_row_bytes_of<E2M1>(HD), N16 = ST::bytes;   // 16-byte pieces
    const int lane = threadIdx.x & 31, g = lane % LPR;
    const int half = (p.num_kv_heads + STEP - 1) / STEP;         // pieces of K; as many of V
    const int gw = blockIdx.x * (kWriteThreads / 32) + (threadIdx.x >> 5);
    const int step = gridDim.x * (kWriteThreads / 32) / (2 * half);
    int64_t t = gw / (2 * half);
    if (t >= step || t >= p.num_tokens) return;
    const int piece = gw % (2 * half);
    const bool v = piece >= half;
    const int h0 = (piece - (v ? half : 0)) * STEP + lane / LPR;
    const uint8_t* src = static_cast<const uint8_t*>(v ? p.value : p.key) + (h0 * HD + 16 * g) * ST::bytes;
    uint8_t* pool = static_cast<uint8_t*>(v ? p.v_cache : p.k_cache);
    const int tile_bytes = p.block_size * TILE_ROW;
    const int64_t src_step = (int64_t)p.num_kv_heads * HD * ST::bytes;
    uint4 now[kWriteRows][N16], next[kWriteRows][N16];
    auto fetch = [&](uint4 (&x)[kWriteRows][N16], int64_t at) {
        const uint4* row = reinterpret_cast<const uint4*>(src + at * src_step);
#pragma unroll
        for (int u = 0; u < kWriteRows; ++u)
#pragma unroll
            for (int i = 0; i < N16; ++i)
                x[u][i] = h0 + u * RPW < p.num_kv_heads ? row[u * (RPW * HD * ST::bytes / 16) + i]
                                                        : make_uint4(0u, 0u, 0u, 0u);
    };
    fetch(now, t);
    int64_t slot = p.slot_mapping[t], slot_next = -1;
    for (; t < p.num_tokens; t += step) {
        if (t + step < p.num_tokens) {
            fetch(next, t + step);
            slot_next = p.slot_mapping[t + step];
        }
        const int64_t blk = slot >> log_block;
        if (slot >= 0 && blk < p.num_blocks) {                   // the whole warp: one token
            const int row = (int)(slot & ((1 << log_block) - 1));
            uint8_t* tile = pool + (blk * p.num_kv_heads + h0) * tile_bytes;
#pragma unroll
            for (int u = 0; u < kWriteRows; ++u) {
                float x[16];
#pragma unroll
                for (int i = 0; i < N16; ++i) Chunk<ST>::to_float(now[u][i], x + i * (16 / N16));
                if (h0 + u * RPW < p.num_kv_heads)
                    CacheRow<E2M1>::store_group(tile + u * RPW * tile_bytes, p.block_size, HD, row, g,
                                                x, p.kv_scale);
            }
        } else if (slot >= 0 && piece == 0 && lane == 0) {
            set_status(p.status, PKV_DEV_BAD_SLOT);
        }
        slot = slot_next;
#pragma unroll
        for (int u = 0; u < kWriteRows; ++u)
#pragma unroll
            for (int i = 0; i < N16; ++i) now[u][i] = next[u][i];
    }
}

// grid = (pairs, slices of a block, 2 caches); one 16-byte chunk per thread-iteration.
// Block pairs[i][0] of the source pool -> block pairs[i][1] of the destination.
__global__ void __launch_bounds__(256) copy_blocks_kernel(CopyParams p) {
    pdl_launch_dependents();
    const int pair = blockIdx.x;
    const int32_t src = p.pairs[2 * pair], dst = p.pairs[2 * pair + 1];
    if (src < 0 || src >= p.src_num_blocks || dst < 0 || dst >= p.dst_num_blocks) {
        if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
            set_status(p.status, PKV_DEV_BAD_PAIR);
        return;
    }
    const uint8_t* sc = static_cast<const uint8_t*>(blockIdx.z == 0 ? p.src_k : p.src_v);
    uint8_t* dc = static_cast<uint8_t*>(blockIdx.z == 0 ? p.dst_k : p.dst_v);
    const uint4* s = reinterpret_cast<const uint4*>(sc + (int64_t)src * p.block_bytes);
    uint4* d = reinterpret_cast<uint4*>(dc + (int64_t)dst * p.block_bytes);
    const int64_t n = p.block_bytes / 16;
    for (int64_t i = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; i < n;
         i += (int64_t)gridDim.y * blockDim.x)
        d[i] = s[i];
}

cudaError_t launch_reshape_and_cache(const ReshapeParams& p, pkv_dtype src, bool quant,
                                     int num_sms, cudaStream_t stream) {
    const int kb = quant ? 1 : (src == PKV_F32 ? 4 : 2);
    const int64_t total = (int64_t)p.num_tokens * p.num_kv_heads * (p.head_dim * kb / 16);
    int64_t want = (total + 255) / 256;
    const int64_t cap = (int64_t)num_sms * 8;
    const int grid = (int)(want < cap ? (want < 1 ? 1 : want) : cap);
    switch (src) {
    case PKV_F32:
        if (quant) reshape_and_cache_kernel<F32, true><<<grid, 256, 0, stream>>>(p);
        else reshape_and_cache_kernel<F32, false><<<grid, 256, 0, stream>>>(p);
        break;
    case PKV_F16:
        if (quant) reshape_and_cache_kernel<F16, true><<<grid, 256, 0, stream>>>(p);
        else reshape_and_cache_kernel<F16, false><<<grid, 256, 0, stream>>>(p);
        break;
    case PKV_BF16:
        if (quant) reshape_and_cache_kernel<BF16, true><<<grid, 256, 0, stream>>>(p);
        else reshape_and_cache_kernel<BF16, false><<<grid, 256, 0, stream>>>(p);
        break;
    default:
        return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

template <typename ST>
static cudaError_t launch_write_fp4(const ReshapeParams& p, int num_sms, cudaStream_t stream) {
    const int step = 512 / p.head_dim * kWriteRows;
    const int64_t pieces = 2 * (int64_t)((p.num_kv_heads + step - 1) / step);
    const int64_t least = (pieces + 7) / 8, need = (p.num_tokens * pieces + 7) / 8;
    const int64_t full = (int64_t)num_sms * kWriteCtas, most = full > least ? full : least;
    const unsigned grid = (unsigned)(need < most ? need : most);
    const int log_block = p.block_size == 8 ? 3 : p.block_size == 16 ? 4 : 5;
    return launch_overlapped(p.head_dim == 128 ? reshape_and_cache_fp4_kernel<ST, 128>
                                               : reshape_and_cache_fp4_kernel<ST, 64>,
                             grid, kWriteThreads, stream, p, log_block);
}

cudaError_t launch_reshape_and_cache_fp4(const ReshapeParams& p, pkv_dtype src, int num_sms,
                                         cudaStream_t stream) {
    if (src == PKV_F32) return launch_write_fp4<F32>(p, num_sms, stream);
    return src == PKV_F16 ? launch_write_fp4<F16>(p, num_sms, stream)
                          : launch_write_fp4<BF16>(p, num_sms, stream);
}

cudaError_t launch_copy_blocks(const CopyParams& p, int num_pairs, cudaStream_t stream) {
    const int64_t chunks = p.block_bytes / 16;
    int slices = (int)((chunks + 255) / 256);
    if (slices > 64) slices = 64;
    if (slices < 1) slices = 1;
    dim3 grid(num_pairs, slices, 2);
    copy_blocks_kernel<<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

// One thread waits on an mbarrier that nothing arrives at: the bounded wait every
// pipeline uses gives up after kWaitNs and the kernel flags PKV_DEV_WAIT_TIMEOUT.
__global__ void wait_bound_probe_kernel(unsigned* status) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
        if (!mbar_wait(&bar, 0)) set_status(status, PKV_DEV_WAIT_TIMEOUT);
    }
}

cudaError_t launch_wait_bound_probe(unsigned* status, cudaStream_t stream) {
    wait_bound_probe_kernel<<<1, 32, 0, stream>>>(status);
    return cudaGetLastError();
}

}  // namespace pkv
