// chunk_attention.cuh -- parameters and launcher of the attention of a chunk of new tokens over a
// paged cache of 16 bits, FP8 or 4 bits, causal or under a sliding window with sinks.
#pragma once

#include "common.cuh"

namespace pkv {

constexpr int kChunkTile = 128;       // rows of a row tile; tokens of a K/V tile ("step")
constexpr int kChunkRows = 256;       // (token, head of the group) rows of an item, at most
constexpr int kChunkMaxCtas = 160;    // persistent CTAs, at most (one an SM)
// Steps that a CTA of a split launch takes at least.
constexpr int kChunkMinRun = 4;
// What splitting costs, in steps of every CTA: two partial states written, the joining kernel.
constexpr int kChunkSplitCost = 8;
// What an item's end costs (its output, the next one's start: 6,000 - 8,000 cycles), in steps.
constexpr int kChunkItemCost = 2;
// Launches of few items plan for themselves, in every CTA's producer warp: a planner in front of them
// costs 5 us (one token 12.9 us with it, 8.1 without; drafts over FP8 98 and 92).  Sequences are one a
// lane.
constexpr int kChunkSelfSeqs = 32;

// (token, head) rows of a sequence and kv head, up to which it goes to the kernel of few rows where a call has
// such sequences (chunk_few_kernel.cuh).
constexpr int kChunkFewRows = 24;
constexpr int kChunkFewShort = 2048;  // tokens that a row sees, up to which one unit an SM is enough for it
// A context that is much longer than the others' share would end long after them, since that kernel does not cut it:
// sequences that walk more than kChunkFewShares times a CTA's share of the few-rows sequences' tokens, and
// kChunkFewAlone more, go to the tile kernel, which cuts them.
constexpr int kChunkFewShares = 3, kChunkFewAlone = 2048;

// A run of an item's steps, as the planner lists them: CTA c's first one is entry c, what else it
// takes (`first`, or the counter) lies behind entry num_ctas - 1.
struct __align__(16) ChunkPiece {
    int s, kvh, pair;                 // sequence, kv head, pair of row tiles
    int j0, j1;                       // its steps
    int slot;                         // partial state it writes, or -1: the whole item is here
    int q_begin, n, ctx;              // the sequence's first row, its rows, its tokens in the cache
    int pad[3];
};

// The item that a CTA begins and another one ends: what the joining kernel needs.
struct __align__(16) ChunkCut {
    int kvh, pair, q_begin, n;
    int last;                         // the CTA with its last steps; below 0: none is left unfinished
    int pad[3];
};

// What the planner leaves besides.
struct __align__(16) ChunkHead {
    int begun;                        // CTAs that have a first piece
    int end;                          // end of the list (whole items: of those behind the first ones)
    int split;                        // a CTA's other pieces are `first`'s, not the counter's
    int next;                         // the counter
    int few_most;                     // tokens that a sequence of few rows walks, at most, to be the other kernel's
    int pad[3];
};

struct ChunkParams {
    const void* q;                    // [total_q, Hq, d]
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;      // [S, max_blocks]
    const int32_t* context_lens;      // [S]: tokens in the cache, the new ones included
    const int32_t* query_start;       // [S + 1]
    void* out;                        // [total_q, Hq, d]
    int* pair_prefix;                 // workspace [S + 1]: pairs of row tiles before a sequence (many sequences)
    ChunkPiece* pieces;               // workspace [max_pieces]
    ChunkCut* cuts;                   // workspace [num_ctas]
    int* first;                       // workspace [kChunkMaxCtas + 1]: a CTA's second piece (split)
    ChunkHead* head;                  // workspace
    float* part_acc;                  // workspace [slots][part_rows][d]
    float2* part_ml;                  // workspace [slots][part_rows]: running max (log2), sum
    unsigned* status;
    int num_seqs, total_q, num_q_heads, num_kv_heads, group, qpt;
    int item_tokens;                  // of an item: qpt (one row tile, NARROW) or 2 qpt
    int block_size, log_block, num_blocks, max_blocks, max_context_len;
    int window, sinks;                // window >= max_context_len: none
    int max_pairs;                    // pairs of row tiles that the workspace has room for
    int num_ctas, part_rows;
    int few_rows;                     // sequences with as many rows of a kv head are another kernel's (0: none)
    int few_ctas;                     // its resident CTAs, where some may be too long for it; else 0
    int self_plan;                    // no planner: every CTA finds its pieces
    int may_split;                    // an item can be cut, by the sizes
    float qk_scale_log2;              // scale * log2(e) * kv_scale
    float out_scale;                  // kv_scale of FP8 and 4 bits, else 1
};

// Sizes of a call's workspace.
struct ChunkPlan {
    int64_t items;                    // at most
    int slots, part_rows, item_tokens;
    size_t off_pieces, off_cuts, off_first, off_head, off_acc, off_ml, total;
};

// What an item sees of its context, and so its steps.  Blocks that none of its rows sees are left out:
// it walks a virtual context, the blocks of the sinks and then, `skip` tokens on, those from the
// window's first one.  Positions count in that context: they keep their order and their distances
// within the window, and its tokens below `low` that are no sinks are seen by no row.  (With the
// sinks' tokens in a tile of their own a window of 1,024 takes 10.5 steps an item instead of 9.)
struct ChunkSpan {
    int skip, sink_blocks, low, kv_end, steps;
};

__host__ __device__ __forceinline__ ChunkSpan chunk_span(int p_first, int kv_end, int window, int sinks,
                                                         int log_block) {
    ChunkSpan w;
    const int past = p_first - window;                 // the last token that the first row does not see
    const int low = past < 0 ? 0 : past + 1;
    const int kept = sinks < low ? sinks : low;
    w.sink_blocks = kept <= 0 ? 0 : ((kept - 1) >> log_block) + 1;
    const int first = low >> log_block;
    w.skip = first > w.sink_blocks ? (first - w.sink_blocks) << log_block : 0;
    w.low = low - w.skip;
    w.kv_end = kv_end - w.skip;
    w.steps = (w.kv_end - 1) / kChunkTile + 1;
    return w;
}

// Whether items are cut into equal runs of q steps, a CTA each, or dealt whole: rounds of items of average length, or
// the longest one, against a run, with as many items' ends as the shortest ones put into it.  (Runs are equal in
// steps: over a prompt's first rows a run holds dozens of short items.  One prompt of 4,096 tokens, 32 / 8 heads, bf16:
// 227 us in runs, 120 whole; 1 x 512 over 8,192 73 in runs, 117 whole.)
__device__ __forceinline__ bool chunk_split(int64_t total, int items, int most, int least, int ctas, int64_t q) {
    if (items == 0) return false;
    const float rounds = (float)((items + ctas - 1) / ctas);
    const float whole = fmaxf((float)most, rounds * ((float)total / (float)items + kChunkItemCost) - kChunkItemCost);
    return whole > (float)q + kChunkSplitCost + (float)q / (float)least * kChunkItemCost;
}

// What a sequence of n rows, the last of ctx tokens, walks, if it has few rows (else 0).
__device__ __forceinline__ int few_tokens(const ChunkParams& p, int64_t n, int ctx) {
    if (n <= 0 || n * p.group > p.few_rows) return 0;
    return chunk_span(ctx - (int)n, ctx, p.window, p.sinks, p.log_block).kv_end;
}

// Tokens that such a sequence walks at most, by what all of them walk.
__device__ __forceinline__ int few_most(const ChunkParams& p, int64_t tokens) {
    if (p.few_ctas == 0) return INT32_MAX;
    return (int)min((int64_t)INT32_MAX, tokens * p.num_kv_heads / p.few_ctas * kChunkFewShares + kChunkFewAlone);
}

// The sum of a warp's lanes.
__device__ __forceinline__ int64_t few_sum(int64_t tokens) {
#pragma unroll
    for (int off = 16; off; off >>= 1) tokens += __shfl_xor_sync(0xffffffffu, tokens, off);
    return tokens;
}

// Defined in chunk_plan.cu.
cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t stream);

// The kernel of few rows, between the planner and the attention: FP8, 4 bits, 16 bits of 64 dims.
cudaError_t chunk_few_f16(const ChunkParams& p, int head_dim, pkv_dtype kv, cudaStream_t s);
cudaError_t chunk_few_bf16(const ChunkParams& p, int head_dim, pkv_dtype kv, cudaStream_t s);

// Attention and joining kernel; each defined in the .cu file of its name.
cudaError_t chunk_f16_16(const ChunkParams& p, int head_dim, cudaStream_t s);
cudaError_t chunk_f16_fp8(const ChunkParams& p, int head_dim, cudaStream_t s);
cudaError_t chunk_f16_fp4(const ChunkParams& p, int head_dim, cudaStream_t s);
cudaError_t chunk_bf16_16(const ChunkParams& p, int head_dim, cudaStream_t s);
cudaError_t chunk_bf16_fp8(const ChunkParams& p, int head_dim, cudaStream_t s);
cudaError_t chunk_bf16_fp4(const ChunkParams& p, int head_dim, cudaStream_t s);

}  // namespace pkv
