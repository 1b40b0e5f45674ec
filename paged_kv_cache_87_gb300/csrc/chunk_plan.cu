// chunk_plan.cu -- the planner of the chunk attention: items into pieces, one CTA.
//
// An item is a (sequence, pair of 128-row tiles, kv head); its steps are the 128-token tiles that
// its rows see.  With items enough for every CTA (one an SM) they are taken whole from a counter,
// sequences with long contexts first.  With few, the flattened steps of all items are cut into
// equal runs, one a CTA, whatever item they belong to; an item that lies in several runs leaves a
// partial state in each, and the joining kernel adds them up in order (no atomics: the same bits
// on every call).  Splitting costs about kChunkSplitCost steps a CTA, whole items cost their last
// round: the cheaper one is taken, by the exact counts.
#include "chunk_attention.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kSortSeqs = 1024;

// Exclusive sum over the block; *total is everything.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* wsum, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t y = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t z = __shfl_up_sync(0xffffffffu, y, off);
        if (lane >= off) y += z;
    }
    if (lane == 31) wsum[warp] = y;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        before += w < warp ? wsum[w] : 0;
        all += wsum[w];
    }
    __syncthreads();
    *total = all;
    return before + y - x;
}

struct Pair {
    int s, pair, steps;
};

// The g-th pair of row tiles in planned order: of a sequence the later (longer) pairs first.
__device__ __forceinline__ Pair pair_at(const ChunkParams& p, int g) {
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {                       // the last sequence whose pairs begin at or before g
        const int mid = (lo + hi + 1) >> 1;
        if (p.pair_prefix[mid] <= g) lo = mid;
        else hi = mid - 1;
    }
    Pair r;
    r.s = p.seq_order[lo];
    r.pair = p.pair_prefix[lo + 1] - 1 - g;
    const int n = p.query_start[r.s + 1] - p.query_start[r.s], ctx = p.context_lens[r.s];
    const int q0 = r.pair * 2 * p.qpt, q1 = min(n, q0 + 2 * p.qpt);
    r.steps = chunk_span(ctx - n + q0, ctx - n + q1, p.window, p.sinks).steps;
    return r;
}

__global__ void __launch_bounds__(kThreads) chunk_plan_kernel(ChunkParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ int64_t wsum[kThreads / 32];
    __shared__ int s_ctx[kSortSeqs];
    __shared__ int s_max;
    const int tid = threadIdx.x;
    if (tid == 0) {
        s_max = 0;
        if (p.query_start[p.num_seqs] != p.total_q || p.query_start[0] != 0)
            set_status(p.status, PKV_DEV_BAD_CONTEXT);
    }
    for (int c = tid; c < kChunkMaxCtas; c += kThreads) p.cuts[c].s = -1;
    // the sequences by context, longest first (a rank sort; beyond kSortSeqs in their order)
    if (p.num_seqs <= kSortSeqs) {
        if (tid < p.num_seqs) s_ctx[tid] = p.context_lens[tid];
        __syncthreads();
        if (tid < p.num_seqs) {
            const int c = s_ctx[tid];
            int rank = 0;
            for (int t = 0; t < p.num_seqs; ++t) rank += s_ctx[t] > c || (s_ctx[t] == c && t < tid);
            p.seq_order[rank] = tid;
        }
    } else {
        for (int s = tid; s < p.num_seqs; s += kThreads) p.seq_order[s] = s;
    }
    __syncthreads();
    // pairs of row tiles before each; a sequence that breaks the contract has none
    const int64_t cap = min((int64_t)p.max_context_len, (int64_t)p.max_blocks * p.block_size);
    int64_t carry = 0;
    for (int base = 0; base < p.num_seqs; base += kThreads) {
        const int k = base + tid;
        int pairs = 0;
        if (k < p.num_seqs) {
            const int s = p.seq_order[k], q0 = p.query_start[s], q1 = p.query_start[s + 1], ctx = p.context_lens[s];
            const int64_t n = (int64_t)q1 - q0;
            if (n < 0 || q0 < 0 || q1 > p.total_q || ctx < n || ctx > cap)
                set_status(p.status, PKV_DEV_BAD_CONTEXT);
            else
                pairs = (int)((n + 2 * p.qpt - 1) / (2 * p.qpt));
        }
        int64_t all;
        const int64_t before = block_scan(pairs, wsum, &all);
        if (k < p.num_seqs) p.pair_prefix[k] = (int)(carry + before);
        carry += all;
    }
    // (starts that run back and forth could list rows twice, and more pairs than there is room for)
    if (carry > p.max_pairs) {
        if (tid == 0) set_status(p.status, PKV_DEV_BAD_CONTEXT);
        carry = 0;
    }
    if (tid == 0) p.pair_prefix[p.num_seqs] = (int)carry;
    __syncthreads();
    const int pairs = (int)carry;
    // all steps, and the longest item's
    int64_t steps = 0;
    int most = 0;
    for (int g = tid; g < pairs; g += kThreads) {
        const int n = pair_at(p, g).steps;
        steps += n;
        most = max(most, n);
    }
    int64_t total;
    block_scan(steps, wsum, &total);
    total *= p.num_kv_heads;
    atomicMax(&s_max, most);
    __syncthreads();
    most = s_max;
    const int64_t items = (int64_t)pairs * p.num_kv_heads;
    const int64_t q = max((int64_t)kChunkMinRun, (total + p.num_ctas - 1) / p.num_ctas);
    // rounds of items of average length, or the longest one
    const int64_t whole = max((int64_t)most, (items + p.num_ctas - 1) / p.num_ctas * total / max(items, (int64_t)1));
    const bool split = whole > q + kChunkSplitCost;
    // the pieces, in the flattened order
    int64_t at_steps = 0, at_pieces = 0;
    for (int base = 0; base < pairs; base += kThreads) {
        const int g = base + tid;
        Pair r{0, 0, 0};
        if (g < pairs) r = pair_at(p, g);
        int64_t all_steps, all_pieces;
        const int64_t pos0 = at_steps + block_scan((int64_t)r.steps * p.num_kv_heads, wsum, &all_steps);
        int64_t mine = 0;
        if (g < pairs) {
            if (split)
                for (int h = 0; h < p.num_kv_heads; ++h) {
                    const int64_t a = pos0 + (int64_t)h * r.steps;
                    mine += (a + r.steps - 1) / q - a / q + 1;
                }
            else
                mine = p.num_kv_heads;
        }
        int64_t i = at_pieces + block_scan(mine, wsum, &all_pieces);
        if (g < pairs)
            for (int h = 0; h < p.num_kv_heads; ++h) {
                ChunkPiece x{r.s, h, r.pair, 0, r.steps, -1, {0, 0}};
                if (!split) {
                    p.pieces[i++] = x;
                    continue;
                }
                const int64_t a = pos0 + (int64_t)h * r.steps, b = a + r.steps;
                const int64_t c0 = a / q, c1 = (b - 1) / q;
                for (int64_t c = c0; c <= c1; ++c) {
                    x.j0 = c == c0 ? 0 : (int)(c * q - a);
                    x.j1 = c == c1 ? r.steps : (int)((c + 1) * q - a);
                    x.slot = c0 == c1 ? -1 : (int)(2 * c + (c == c0));
                    if ((a + x.j0) % q == 0) p.first[c] = (int)i;
                    p.pieces[i++] = x;
                }
                if (c0 != c1) p.cuts[c0] = ChunkCut{r.s, h, r.pair, (int)c1};
            }
        at_steps += all_steps;
        at_pieces += all_pieces;
    }
    if (tid == 0) {
        const int64_t used = split ? (total + q - 1) / q : 0;     // CTAs with work
        for (int64_t c = used; c <= p.num_ctas; ++c) p.first[c] = (int)at_pieces;
        p.head[0] = (int)at_pieces;
        p.head[1] = split;
        p.head[2] = 0;
    }
}

}  // namespace

cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t stream) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, chunk_plan_kernel, p);
}

}  // namespace pkv
