// chunk_plan.cu -- the planner of the chunk attention: items into pieces, one CTA.
//
// An item is a (sequence, pair of 128-row tiles, kv head); its steps are the 128-token tiles that
// its rows see.  With items enough for every CTA (one an SM) they are taken whole from a counter,
// sequences with long contexts first.  With few, the flattened steps of all items are cut into
// equal runs, one a CTA, whatever item they belong to; an item that lies in several runs leaves a
// partial state in each, and the joining kernel adds them up in order (no atomics: the same bits
// on every call).  Splitting costs about kChunkSplitCost steps a CTA, whole items cost their last
// round: the cheaper one is taken (chunk_split), by the exact counts.
//
// Its time is latency, in front of every call: lengths and starts are read once, and up to kSeqs
// sequences everything after that is in shared memory.
#include "chunk_attention.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kSeqs = 1024;            // sequences that are ranked, and planned in shared memory

// Exclusive sum over the block; *total is everything.  (No barrier before: wsum must be free.)
__device__ __forceinline__ int block_scan(int x, int* wsum, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, off);
        if (lane >= off) y += z;
    }
    if (lane == 31) wsum[warp] = y;
    __syncthreads();
    int w = wsum[lane];                // every warp adds the warps' sums up for itself
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += z;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return (warp ? before : 0) + y - x;
}

// The sequence planned k-th: its index, first row, rows, and tokens in the cache.
struct Seq {
    int s, q0, n, ctx;
};

// Steps of the g-th pair of row tiles in planned order (of a sequence the later, longer pairs first).
struct Pair {
    Seq q;
    int pair, steps;
};

__global__ void __launch_bounds__(kThreads) chunk_plan_kernel(ChunkParams p) {
    pdl_launch_dependents();
    __shared__ int wsum[2][32];
    __shared__ int s_ctx[kSeqs];
    __shared__ Seq s_seq[kSeqs];
    __shared__ int s_prefix[kSeqs + 1];
    __shared__ int s_most, s_least;
    __shared__ unsigned long long s_total, s_few;
    const int tid = threadIdx.x, S = p.num_seqs;
    const bool small = S <= kSeqs;
    if (tid == 0) {
        s_most = 0;
        s_least = INT32_MAX;
        s_total = 0;
        s_few = 0;
    }
    pdl_wait();
    for (int c = tid; c < p.num_ctas; c += kThreads) p.cuts[c].last = -1;
    const int64_t cap = min((int64_t)p.max_context_len, (int64_t)p.max_blocks * p.block_size);
    auto good = [&](int q0, int q1, int ctx) {
        const int64_t n = (int64_t)q1 - q0;
        return n >= 0 && q0 >= 0 && q1 <= p.total_q && ctx >= n && ctx <= cap;
    };
    int few = INT32_MAX;
    if (p.few_ctas) {                       // which sequences of few rows are too long for their kernel
        unsigned long long tokens = 0;
        for (int s = tid; s < S; s += kThreads) {
            const int q0 = p.query_start[s], q1 = p.query_start[s + 1], ctx = p.context_lens[s];
            if (good(q0, q1, ctx)) tokens += few_tokens(p, (int64_t)q1 - q0, ctx);
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) tokens += __shfl_xor_sync(0xffffffffu, tokens, off);
        __syncthreads();
        if ((tid & 31) == 0 && tokens) atomicAdd(&s_few, tokens);
        __syncthreads();
        few = few_most(p, (int64_t)s_few);
    }
    // pairs of a sequence; one that breaks the contract, or is another kernel's, has none
    auto pairs_of = [&](int q0, int q1, int ctx) {
        const int64_t n = (int64_t)q1 - q0;
        if (good(q0, q1, ctx))
            return n * p.group <= p.few_rows && few_tokens(p, n, ctx) <= few
                       ? 0 : (int)(((uint32_t)n + p.item_tokens - 1) / (uint32_t)(p.item_tokens));
        set_status(p.status, PKV_DEV_BAD_CONTEXT);
        return 0;
    };
    if (tid == 0 && (p.query_start[S] != p.total_q || p.query_start[0] != 0))
        set_status(p.status, PKV_DEV_BAD_CONTEXT);
    int64_t carry = 0;
    if (small) {
        // by context, longest first (a rank sort); then prefix sums of the pairs
        Seq me{tid, 0, 0, 0};
        int q1 = 0;
        if (tid < S) {
            me.q0 = p.query_start[tid];
            q1 = p.query_start[tid + 1];
            me.ctx = p.context_lens[tid];
            s_ctx[tid] = me.ctx;
        }
        __syncthreads();
        if (tid < S) {
            me.n = pairs_of(me.q0, q1, me.ctx) ? q1 - me.q0 : 0;
            int rank = 0;
            for (int t = 0; t < S; ++t) {
                const int c = s_ctx[t];
                rank += c > me.ctx || (c == me.ctx && t < tid);
            }
            s_seq[rank] = me;
        }
        __syncthreads();
        const int pairs = tid < S ? (s_seq[tid].n + p.item_tokens - 1) / (p.item_tokens) : 0;
        int all;
        s_prefix[tid] = block_scan(pairs, wsum[0], &all);
        carry = all;
    } else {
        for (int base = 0; base < S; base += kThreads) {
            const int s = base + tid;
            const int pairs = s < S ? pairs_of(p.query_start[s], p.query_start[s + 1], p.context_lens[s]) : 0;
            int all;
            const int before = block_scan(pairs, wsum[0], &all);
            if (s < S) p.pair_prefix[s] = (int)min(carry + before, (int64_t)INT32_MAX);
            carry += all;
            __syncthreads();
        }
    }
    // (starts that run back and forth could list rows twice, and more pairs than there is room for)
    if (carry > p.max_pairs) {
        if (tid == 0) set_status(p.status, PKV_DEV_BAD_CONTEXT);
        carry = 0;
    }
    const int pairs = (int)carry;
    if (tid == 0) {
        if (small) s_prefix[S] = pairs;
        else p.pair_prefix[S] = pairs;
    }
    __syncthreads();
    auto pair_at = [&](int g) {
        const int* prefix = small ? s_prefix : p.pair_prefix;
        int lo = 0, hi = S - 1;
        while (lo < hi) {                   // the last sequence whose pairs begin at or before g
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= g) lo = mid;
            else hi = mid - 1;
        }
        Pair r;
        if (small) {
            r.q = s_seq[lo];
        } else {
            r.q.s = lo;
            r.q.q0 = p.query_start[lo];
            r.q.n = p.query_start[lo + 1] - r.q.q0;
            r.q.ctx = p.context_lens[lo];
        }
        r.pair = prefix[lo + 1] - 1 - g;
        const int a = r.pair * p.item_tokens, b = min(r.q.n, a + p.item_tokens), before = r.q.ctx - r.q.n;
        r.steps = chunk_span(before + a, before + b, p.window, p.sinks, p.log_block).steps;
        return r;
    };
    // all steps, the longest item's and the shortest one's
    int64_t steps = 0;
    int most = 0, least = INT32_MAX;
    for (int g = tid; g < pairs; g += kThreads) {
        const int n = pair_at(g).steps;
        steps += n;
        most = max(most, n);
        least = min(least, n);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) steps += __shfl_xor_sync(0xffffffffu, steps, off);
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if ((tid & 31) == 0 && most) {
        atomicAdd(&s_total, (unsigned long long)steps);
        atomicMax(&s_most, most);
        atomicMin(&s_least, least);
    }
    __syncthreads();
    most = s_most;
    const int64_t total = (int64_t)s_total * p.num_kv_heads, items = (int64_t)pairs * p.num_kv_heads;
    const int64_t q64 = max((int64_t)kChunkMinRun, (total + p.num_ctas - 1) / p.num_ctas);
    const bool split = chunk_split(total, (int)items, most, s_least, p.num_ctas, q64) && total <= INT32_MAX - (1 << 20);
    const uint32_t q = (uint32_t)q64;
    // the pieces, in the flattened order, an item a thread
    const int nitems = (int)items, used = split ? (int)((total + q - 1) / q) : min(nitems, p.num_ctas);
    int at_steps = 0, extras = 0;
    for (int base = 0; base < nitems; base += kThreads) {
        const int i = base + tid, h = i % p.num_kv_heads;
        Pair r{};
        if (i < nitems) r = pair_at(i / p.num_kv_heads);
        ChunkPiece x{r.q.s, h, r.pair, 0, r.steps, -1, r.q.q0, r.q.n, r.q.ctx, {0, 0, 0}};
        if (!split) {
            if (i < nitems) p.pieces[i] = x;
            continue;
        }
        int all_steps, all_extras;
        const uint32_t a = at_steps + block_scan(r.steps, wsum[0], &all_steps), b = a + r.steps;
        const uint32_t c0 = a / q, c1 = i < nitems ? (b - 1) / q : 0;
        const bool extra = i < nitems && a != c0 * q;        // its first piece is not its CTA's first
        int e = extras + block_scan(extra, wsum[1], &all_extras);
        if (i < nitems) {
            if (extra) {
                x.j1 = min(r.steps, (int)((c0 + 1) * q - a));
                x.slot = c0 == c1 ? -1 : (int)(2 * c0 + 1);
                p.pieces[p.num_ctas + e++] = x;
            }
            for (uint32_t c = c0 + extra; c <= c1; ++c) {
                x.j0 = (int)(c * q - a);
                x.j1 = min(r.steps, (int)((c + 1) * q - a));
                x.slot = c0 == c1 ? -1 : (int)(2 * c + (c == c0));
                p.pieces[c] = x;
                p.first[c] = p.num_ctas + e;
            }
            if (c0 != c1) p.cuts[c0] = ChunkCut{h, r.pair, r.q.q0, r.q.n, (int)c1, {0, 0, 0}};
        }
        at_steps += all_steps;
        extras += all_extras;
        __syncthreads();
    }
    for (int c = tid; c <= p.num_ctas; c += kThreads)        // where CTAs without work would begin
        if (c >= used) p.first[c] = p.num_ctas + extras;
    if (tid == 0) *p.head = ChunkHead{used, split ? p.num_ctas + extras : nitems, split, p.num_ctas, few, {0, 0, 0}};
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
