// decode_fp4.cuh -- parameters and host launcher of the decode over the 4-bit cache.
#pragma once

#include "common.cuh"
#include "window_span.cuh"

namespace pkv {

constexpr int kFp4Tile = 128;         // tokens of a tile: the split's unit and a ring stage
// Slots of a unit besides its tiles (a serving batch takes 141 us with 0, 103.5 with 1, 104.6 with 2).
constexpr int kFp4UnitCost = 1;
// Slots a worker takes at least (one context of 600 tokens: 8.0 us with 1, 8.7 with 2).
constexpr int kFp4MinQuota = 1;
// Partial states that one unit leaves, about (one context of 100,000 tokens and one kv head: 95 us
// without a bound, 22 with 64 or 128, 29 with 32).
constexpr int kFp4MaxPieces = 64;
constexpr int kFp4MaxWorkers = 1024;  // CTAs of the decode, at most (half with units of 16 heads)

// Query heads of a work unit: one kv head's group, in parts of 16 at most.  Groups of up to eight
// take the kernel whose unit is eight (long documents: 151 us at eight heads a group; at sixteen,
// 228 us in one unit, and 233 against 307 in two when that was chosen).
inline int fp4_unit_heads(int group) { return group > 8 ? 16 : 8; }

// Few short contexts: a cluster of up to eight CTAs takes a unit and joins it by itself -- the largest
// size, not above the tiles, with which every unit's cluster is resident at once, if no CTA has more than
// kFp4ClusterTiles tiles then (eight, in clusters of eight; what a longer run of one CTA costs outweighs the
// joining kernel).  Measured (us, clusters against equal runs and a joining kernel), 32 / 8 heads, d 128:
// one sequence of 100 tokens 5.0 against 6.7, 600 6.3 against 8.1, 2,000 7.2 against 9.4, 8,192 11.5 against
// 11.8; 14 sequences of 100 5.5 against 7.9, 600 9.1 against 11.2, 1 - 1,000 8.7 against 9.4.  Without the
// bound on tiles, 20 sequences of 1 - 2,000: 15.4 against 10.9; without that on residence, 7 of 4,096: 21
// against 17.
constexpr int kFp4Cluster = 8;        // CTAs of a cluster, at most (a power of two)
constexpr int kFp4ClusterTiles = 4;

struct DecodeFp4Params {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    void* out;
    unsigned* status;
    float* part_acc;       // [workers * 2][unit_heads][head_dim]
    float* part_ml;        // [workers * 2][unit_heads][2]: running max (log2 domain) and sum
    int4* cuts;            // [workers]: {1, sequence, unit, its last worker} of a unit it began and
                           // left unfinished, or {0}
    int num_seqs, num_q_heads, num_kv_heads, group, nsub, unit_heads;
    int head_dim, block_size, num_blocks, max_blocks;
    int max_context_len;   // at most max_blocks * block_size
    int window, sinks;     // sliding window and first tokens that stay visible (0: no window)
    int max_seen;          // tokens of a virtual context (window_span.cuh), at most; else max_context_len
    int log_block;         // block_size == 1 << log_block
    int workers;           // the split's denominator: every CTA the device holds
    int max_workers;       // workers that can have work, by max_context_len
    int log_cluster;       // of the CTAs of a unit's cluster
    float qk_scale_log2;   // scale * log2(e) * kv_scale
    float out_scale;       // kv_scale
    uint32_t even, odd, minus;     // 2^4 + 2^16, 1 + 2^12, -1: shifts as products
};

// Workers that can have work over contexts up to max_ctx: bounds grid and workspace.
inline int64_t fp4_max_workers(int num_seqs, int num_kv_heads, int nsub, int unit_heads,
                               int max_ctx) {
    const int64_t slots = (int64_t)num_seqs * num_kv_heads * nsub *
                          (((int64_t)max_ctx + kFp4Tile - 1) / kFp4Tile + kFp4UnitCost);
    const int64_t w = (slots + kFp4MinQuota - 1) / kFp4MinQuota;
    const int64_t most = kFp4MaxWorkers * 8 / unit_heads;
    return w < 1 ? 1 : (w < most ? w : most);
}

// Defined in decode_fp4_f32.cu, decode_fp4_f16.cu and decode_fp4_bf16.cu.
cudaError_t decode_fp4_f32(const DecodeFp4Params& p, cudaStream_t s);
cudaError_t decode_fp4_f16(const DecodeFp4Params& p, cudaStream_t s);
cudaError_t decode_fp4_bf16(const DecodeFp4Params& p, cudaStream_t s);

// The same under a sliding window (decode_fp4_window_*.cu): fp32 queries, and wide windows.  16-bit
// queries over virtual contexts of up to kFp4WindowMost tokens take decode_window_kernel.cuh.  Measured
// (us, that kernel | this one), 32 / 8 heads, d 128: under a window of 1,024, 1, 16, 64 and 256 sequences 5.8 | 8.1,
// 10.3 | 13.4, 22.1 | 27.1, 70.8 | 82.5; of 2,000 6.3 | 8.2, 14.3 | 16.7, 38.9 | 38.8, 126 | 124; of 2,500 6.9 | 8.9,
// 16.5 | 18.3, 47.5 | 44.3, 155 | 147; of 8,192 10.6 | 12.5, 40.8 | 36.6, 148 | 118, 474 | 430.  Of 64 dims the two meet
// earlier where there are many: 1,024 5.7 | 7.3, 12.0 | 9.8, 18.0 | 19.9, 51.8 | 48.2; 2,000 6.2 | 7.5, 14.6 | 11.7,
// 28.9 | 27.1, 93.0 | 76.2.
constexpr int kFp4WindowMost = 2048;
cudaError_t decode_fp4_window_f32(const DecodeFp4Params& p, cudaStream_t s);
cudaError_t decode_fp4_window_f16(const DecodeFp4Params& p, cudaStream_t s);
cudaError_t decode_fp4_window_bf16(const DecodeFp4Params& p, cudaStream_t s);

}  // namespace pkv
