// gather.cu -- rows of the paged cache read back into contiguous K and V rows.
//
// out[r] = value of token (r - row_start[s] + token_start[s]) of the sequence s whose run
// holds r: a pure copy (16- and 32-bit caches) or code * scale * kv_scale (FP8, 4 bits).
// Bound by HBM: 2 * heads * d * (cache bytes + out bytes) per row.  Measured from 4 bits: 48 contexts,
// 154 thousand rows to fp16 119 us (6.65 TB/s, 0.98 of the measured copy rate), one context of 5,000
// tokens to bf16 5.7 us (0.68).
//
// A CTA takes kGatherRows consecutive output rows (8: more CTAs for short runs; 32 took 7.5 us on the
// one context and 123 us on the 48).  One thread per row finds its sequence (binary search in
// row_start) and its place in the pool; then every warp takes the rows of one kv head at a time,
// four lanes to a row with every load of it in flight, so that eight consecutive tokens of a block
// read whole 128-byte lines of 4-bit codes and write 64-byte runs.
#include "cache_ops.cuh"
#include "cache_row.cuh"

namespace pkv {

constexpr int kGatherRows = 8;
constexpr int kGatherThreads = 256;

template <typename KT, typename OT, int HD>
__global__ void __launch_bounds__(kGatherThreads) gather_cache_kernel(GatherParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ int64_t s_place[kGatherRows];   // block * block_size + row in it, or -1
    const int r0 = blockIdx.x * kGatherRows;
    const int n = min(kGatherRows, p.total_rows - r0);
    const int B = p.block_size;
    if (threadIdx.x < kGatherRows) {
        int64_t place = -1;
        const int r = r0 + threadIdx.x;
        if (threadIdx.x < n) {
            // the last sequence starting at or before r
            int lo = 0, hi = p.num_seqs - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.row_start[mid] <= r) lo = mid;
                else hi = mid - 1;
            }
            const int first = p.row_start[lo];
            if (first <= r && r < p.row_start[lo + 1]) {
                const int64_t tok = (int64_t)(p.token_start ? p.token_start[lo] : 0) + (r - first);
                if (tok < 0 || tok >= (int64_t)p.max_blocks * B) {
                    set_status(p.status, PKV_DEV_BAD_CONTEXT);
                } else {
                    const int blk = p.block_tables[(int64_t)lo * p.max_blocks + tok / B];
                    if (blk < 0 || blk >= p.num_blocks) set_status(p.status, PKV_DEV_BAD_BLOCK_ID);
                    else place = (int64_t)blk * B + tok % B;
                }
            }
        }
        s_place[threadIdx.x] = place;
    }
    __syncthreads();
    constexpr int kGroups = kGatherRows / 8;
    const int lane = threadIdx.x & 31, sub = lane >> 2, w = lane & 3;
    const int64_t tile_bytes = (int64_t)B * cache_row_bytes_of<KT>(HD);
    const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache);
    const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache);
    for (int it = threadIdx.x >> 5; it < kGroups * p.num_kv_heads; it += kGatherThreads / 32) {
        const int h = it / kGroups, i = (it % kGroups) * 8 + sub;
        const int64_t place = s_place[i];
        if (place < 0) continue;
        const int row = (int)(place % B);
        const int64_t tile = (place / B * p.num_kv_heads + h) * tile_bytes;
        const int64_t dst = ((int64_t)(r0 + i) * p.num_kv_heads + h) * HD * OT::bytes;
        typename CacheRow<KT>::template Raw<HD> rk, rv;       // every load first
        CacheRow<KT>::template fetch<HD>(kc + tile, B, row, w, rk);
        CacheRow<KT>::template fetch<HD>(vc + tile, B, row, w, rv);
        uint8_t* ko = static_cast<uint8_t*>(p.key_out) + dst;
        uint8_t* vo = static_cast<uint8_t*>(p.value_out) + dst;
        if constexpr (!is_quantised<KT>()) {
            CacheRow<KT>::template copy<HD>(rk, w, ko);
            CacheRow<KT>::template copy<HD>(rv, w, vo);
        } else {
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) {
                const int j = 4 * c + w;
                float k[8], v[8];
                CacheRow<KT>::template values<HD>(rk, c, w, k);
                CacheRow<KT>::template values<HD>(rv, c, w, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    k[e] *= p.kv_scale;
                    v[e] *= p.kv_scale;
                }
                store8<OT>(ko + j * 8 * OT::bytes, k);
                store8<OT>(vo + j * 8 * OT::bytes, v);
            }
        }
    }
}

template <typename KT, typename OT>
cudaError_t launch_gather(const GatherParams& p, cudaStream_t stream) {
    const int64_t grid = ((int64_t)p.total_rows + kGatherRows - 1) / kGatherRows;
    return launch_overlapped(p.head_dim == 128 ? gather_cache_kernel<KT, OT, 128>
                                               : gather_cache_kernel<KT, OT, 64>,
                             (unsigned)grid, kGatherThreads, stream, p);
}

cudaError_t launch_gather_cache(const GatherParams& p, pkv_dtype kv, pkv_dtype out,
                                cudaStream_t stream) {
    if (kv == PKV_FP4_E2M1) {
        if (out == PKV_F32) return launch_gather<E2M1, F32>(p, stream);
        return out == PKV_F16 ? launch_gather<E2M1, F16>(p, stream)
                              : launch_gather<E2M1, BF16>(p, stream);
    }
    if (kv == PKV_FP8_E4M3) {
        if (out == PKV_F32) return launch_gather<E4M3, F32>(p, stream);
        return out == PKV_F16 ? launch_gather<E4M3, F16>(p, stream)
                              : launch_gather<E4M3, BF16>(p, stream);
    }
    if (kv == PKV_F32) return launch_gather<F32, F32>(p, stream);
    return kv == PKV_F16 ? launch_gather<F16, F16>(p, stream) : launch_gather<BF16, BF16>(p, stream);
}

}  // namespace pkv
