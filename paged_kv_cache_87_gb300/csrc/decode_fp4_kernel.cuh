// decode_fp4_kernel.cuh -- single-query decode attention over the 4-bit paged cache.
//
// o = sum_t softmax_t(scale q.k_t) v_t with k, v = code * scale * kv_scale; kv_scale is folded
// into the logit scale and the output.
//
// Products.  code * scale has at most 2 + 4 significant bits and lies in [2^-10, 2688]: it is
// exact in fp16, so a widening convert and one packed multiply make tensor-core operands of
// the stored bytes without a rounding (mma.sync m16n8k16, fp32 accumulation):
//   S^T[16 tokens x 8 heads] = K[16 x d] . Q^T        O^T[d x 8] += V^T[d x 16] . P^T[16 x 8]
// Queries of any type become fp16 exactly enough: each head's row is scaled by a power of two
// that puts its largest magnitude in [2^14, 2^15) (undone in the logit scale), so a 16-bit row
// keeps every bit down to 2^-39 of its largest value.  fp32 queries take two such terms (22
// bits).  Weights enter the second product as fp16 in [0, 2^15] (they are taken 2^7 above the running
// maximum, which is moved when the sum of a lane's two or four passes 2^15, so that a weight 2^-31 of
// the largest still counts), for fp32 queries as two terms of them in [0, 60000] (2^13 above, down to
// 2^-37); the denominator sums them in fp32 before that rounding, and what is smaller still counts
// there alone: n tokens lose at most n 2^-32 of an output (n 2^-38).
//
// Layout.  32 dims of a row are 16 bytes, eight rows of them one 128-byte line: ldmatrix reads
// them free of bank conflicts with no swizzle, and one gather moves 32 or 64 tokens of K or V, codes
// and scales.  A lane's 4-byte word of K holds dims 8c .. 8c + 7 of row g: its four bytes
// are four operand pairs, the reduction index being permuted for K and q alike.  A transposed
// word of V holds dims 4g .. 4g + 3 of tokens 2c and 2c + 1: a mask and three products (as shifts)
// pair the tokens' nibbles in bytes.  (Leaving the pairs of dims as they are and giving each of the
// two a product with zeros in the weights saves those and costs eight more mma: 163 us against 160 on
// long documents, 252 against 233 with sixteen heads; pairing after the conversion, by byte
// permutations: 165 against 158.)
//
// Split.  Every (sequence, kv head, 8 or 16 query heads) unit is cut into 128-token tiles, and the
// flattened tiles are dealt in equal runs to one CTA each ("worker"), all resident at once.
// Every CTA derives the plan by itself from context_lens (a block-wide scan), so no planning
// kernel runs first.  A CTA is a producer warp, which plans 32 tiles at a time, one a lane, and
// fills a ring of them, and four consumer warps, 2 x 16 tokens of every tile each, whose states
// meet in shared memory at the end of a unit.  Units inside one run are written straight to `out`; a
// worker leaves at most two partial states (its first and its last unit), and merge_fp4_kernel
// joins those of each cut unit in order.  Few short contexts take a cluster a unit instead, whose
// CTAs join their states themselves.
//
// What bounds it.  The consumers' instructions, not HBM: 275 for 16 tokens of K and V at head_dim 128
// (128 of them the converts and multiplies), issued at 2.4 a clock an SM; and 3 - 4 us
// that the joining of the cut units takes after the last of them.  Without the
// arithmetic the same kernel streams at 0.97 of the copy rate.  Measured (device time, GB300):
//   long documents (8 x 32k - 131k tokens, 64 / 8 heads, d 128, blocks of 32): 151 us, 5.70 TB/s,
//     0.84 of the measured copy rate; a first, CUDA-core kernel 14,124 us
//   serving batch (256 x 64 - 8k, 32 / 8 heads, d 128, blocks of 16): 104 us, 4.86 TB/s, 0.72
//   ragged (67 x 1 - 4k, 20 / 20 heads, d 64, blocks of 8): 26.6 us, 2.29 TB/s, 0.34: the units are
//     short, and one costs 0.8 of a tile besides its tiles
//   one context of 600 tokens: 6.3 us, latency (8.1 in equal runs with a joining kernel)
//   sixteen query heads a kv head (long documents of 842 MB): 223 us, 0.56; fp32 queries over them: 204 us,
//     0.61: twice the products for the same rows
// Tried and not kept (each against the step of its time): four warps loading their own tokens by
// 16-byte asynchronous copies, without a producer (237 against 160 us on long documents); no producer,
// the last warp through with a stage filling it again (186 against 158); operands of q in registers
// (187 against 175); a fifth CTA a SM at 72 registers (200 against 175); one piece of 16 tokens a warp
// at a time (167 against 158; with four CTAs 164); two stages (164 against 158); halves of the loops
// rolled up (168 - 172 against 160).
#pragma once

#include "decode_fp4.cuh"

#include "cache_row.cuh"
#include "cluster.cuh"
#include "tmap.cuh"

namespace pkv {
namespace {

// Four rows of a 2-D tensor by their indices into consecutive rows of shared memory.
__device__ __forceinline__ void tma_gather4(void* smem_dst, const CUtensorMap* map, int y0, int y1,
                                            int y2, int y3, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;"
        ::"r"(smem_addr(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y0), "r"(y1),
        "r"(y2), "r"(y3), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

__device__ __forceinline__ uint32_t trans8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
        "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// What is left of (lo, hi) after pack_f16's rounding, as fp16 again.
__device__ __forceinline__ uint32_t pack_f16_rest(float lo, float hi, uint32_t packed) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&packed));
    return pack_f16(lo - v.x, hi - v.y);
}

// Weights are 2^(x - m + kLift) with the running maximum m, which moves to a larger logit where a
// lane's weights of a head sum to more than kMost: one of the two or four is kSlack (log2) past m
// then, and below kMost no weight leaves fp16.  fp32 queries keep more of what is far below the
// largest weight (down to 2^-38 of it instead of 2^-32) and move the maximum more often.
template <typename QT>
struct Weight {
    static constexpr float kLift = 7.f, kMost = 32768.f, kSlack = 5.5f;   // 2^(15 - 2 - 7) > 2^5.5
};
template <>
struct Weight<F32> {
    static constexpr float kLift = 13.f, kMost = 60000.f, kSlack = 0.8f;  // 60000 / 4 > 2^(13 + 0.8)
};
constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);

// NT: groups of eight query heads that a unit serves (each widened row of K and V serves them all)
template <typename QT, int HD, int NT>
struct Cfg {
    static constexpr int HEADS = 8 * NT;
    static constexpr int ROWB = HD / 2 + HD / 16;
    static constexpr int KV_BYTES = kFp4Tile * ROWB;
    static constexpr int Q_BYTES = HEADS * HD * QT::bytes;
    static constexpr int STAGE_BYTES = (2 * KV_BYTES + Q_BYTES + 127) / 128 * 128;
    static constexpr int NSTAGE = 3;
    static constexpr int NCHUNK = HD / 32;
    static constexpr int NP = std::is_same<QT, F32>::value ? 2 : 1;   // terms of q and p
    static constexpr int XD = 64;                      // dims of eight heads exchanged at a time
    static constexpr int HS = XD + 1;                  // exchange stride of a head: few conflicts
    static constexpr int XBUF = kConsumers * (8 * HS + 2 * HEADS);    // acc, then m, l
    static constexpr size_t OFF_META = (size_t)NSTAGE * STAGE_BYTES;
    static constexpr size_t OFF_BARS = OFF_META + NSTAGE * 16;
    static constexpr size_t OFF_QF = (OFF_BARS + 2 * NSTAGE * 8 + 15) / 16 * 16;
    static constexpr size_t OFF_PLAN = OFF_QF + NP * NT * NCHUNK * 32 * 16;  // 32 tiles: int4, int2, rows
    static constexpr size_t OFF_X = OFF_PLAN + 32 * (16 + 8 + 16 * 4);
    static constexpr size_t SMEM = OFF_X + XBUF * 4 + 128;             // the base is rounded up
    static_assert(HEADS * (HD + 2) * 4 <= STAGE_BYTES, "a stage holds a CTA's state");
    // resident CTAs, by registers
    static constexpr int CTAS = HD == 128 ? (NT == 1 ? 3 : 2) : (NT == 1 ? 4 : 3);
    // pieces of 16 tokens a warp works on at once, by registers
    static constexpr int PIECES = NT == 1 ? 2 : 1;
};

constexpr int kFirst = 1, kLast = 2, kDone = 4;

// Tokens of a tile, from the first word of its record.
template <bool WIN>
__device__ __forceinline__ int tile_tokens(int x) { return WIN ? x >> 8 & 255 : x >> 8; }

// The hidden tokens of a tile of sequence s, in the bits of that word: [first, end).
__device__ __forceinline__ int hidden_of(const DecodeFp4Params& p, int s, int tile) {
    const WindowSpan w = window_span(min(p.context_lens[s], p.max_context_len), p.window, p.sinks, p.log_block);
    const int lo = min(max(w.hide_lo - tile * kFp4Tile, 0), kFp4Tile);
    const int hi = min(max(w.hide_hi - tile * kFp4Tile, 0), kFp4Tile);
    return (int)((uint32_t)lo << 16 | (uint32_t)hi << 24);
}

// Tokens of a sequence's context that are walked: under a window (WIN) its virtual context's.
template <bool WIN>
__device__ __forceinline__ int tokens_of(const DecodeFp4Params& p, int s) {
    const int n = min(p.context_lens[s], p.max_context_len);
    if constexpr (WIN) return n <= 0 ? 0 : window_span(n, p.window, p.sinks, p.log_block).tokens;
    return n;
}

// Tiles of a sequence's context, per unit.
template <bool WIN>
__device__ __forceinline__ int tiles_of(const DecodeFp4Params& p, int s) {
    const int n = tokens_of<WIN>(p, s);
    return n <= 0 ? 0 : (n - 1) / kFp4Tile + 1;          // (n + 127 would pass 31 bits)
}

// A unit's length in the plan, in slots: its tiles and, before them, kFp4UnitCost slots that
// stand for what a unit costs besides (its queries, the warps' meeting at its end).
template <bool WIN>
__device__ __forceinline__ int slots_of(const DecodeFp4Params& p, int s) {
    const int n = tiles_of<WIN>(p, s);
    return n ? n + kFp4UnitCost : 0;
}

// Block-wide scan of the sequences' slots: pref[i] = slots of the sequences before thread i's run
// of ceil(S / threads), pref[threads] = all, pref[threads + 1] = the longest.  Syncs the block.
template <int THREADS, bool WIN>
__device__ __forceinline__ void scan_slots(const DecodeFp4Params& p, int* pref, int2* wsum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int run = (p.num_seqs + THREADS - 1) / THREADS;
    int n = 0, most = 0;
    for (int s = tid * run; s < min(p.num_seqs, (tid + 1) * run); ++s) {
        const int k = slots_of<WIN>(p, s);
        n += k;
        most = max(most, k);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    int x = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) wsum[warp] = make_int2(x, most);
    __syncthreads();
    int before = 0;
    most = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const int2 v = wsum[w];
        before += w < warp ? v.x : 0;
        most = max(most, v.y);
    }
    pref[tid + 1] = before + x;
    if (tid == 0) {
        pref[0] = 0;
        pref[THREADS + 1] = most;
    }
    __syncthreads();
}

// Place of flattened slot `pos` (below the total): its sequence, that sequence's slots a unit, and
// the position of the sequence's first slot.
template <int THREADS, bool WIN>
__device__ __forceinline__ void locate(const DecodeFp4Params& p, const int* pref, int upi, int pos,
                                       int* seq, int* slots, int* base) {
    int lo = 0, hi = THREADS - 1;
    while (lo < hi) {                       // the last run starting at or before pos
        const int mid = (lo + hi + 1) >> 1;
        if (pref[mid] * upi <= pos) lo = mid;
        else hi = mid - 1;
    }
    const int run = (p.num_seqs + THREADS - 1) / THREADS;
    int s = lo * run, b = pref[lo] * upi, n = slots_of<WIN>(p, s);
    while (b + n * upi <= pos) {
        b += n * upi;
        n = slots_of<WIN>(p, ++s);
    }
    *seq = s;
    *slots = n;
    *base = b;
}

// Slots of a worker: an equal share, not under the least that pays, and not so few that one unit
// leaves more than kFp4MaxPieces partial states to join.
__device__ __forceinline__ int quota_of(const DecodeFp4Params& p, int total, int longest) {
    return max(max(kFp4MinQuota, (total + p.workers - 1) / p.workers),
               (longest + kFp4MaxPieces - 1) / kFp4MaxPieces);
}

// CLUSTER: a cluster of 1 << p.log_cluster CTAs takes one unit, a run of its tiles each, and joins its
// own states through distributed shared memory (a lone CTA writes its unit straight to `out`).
// WIN: contexts under a sliding window: the tiles are those of the virtual contexts of window_span.cuh,
// and the hidden tokens in them are masked like those past the context.
template <typename QT, int HD, int NT, bool CLUSTER, bool WIN>
__global__ void __launch_bounds__(kThreads, (Cfg<QT, HD, NT>::CTAS))
    decode_fp4_kernel(DecodeFp4Params p, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
    using C = Cfg<QT, HD, NT>;
    constexpr float kLift = Weight<QT>::kLift, kMost = Weight<QT>::kMost, kSlack = Weight<QT>::kSlack;
    constexpr int HEADS = C::HEADS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_addr(smem_raw) & 127u);
    __shared__ int s_pref[kThreads + 2];
    __shared__ int2 s_wsum[kThreads / 32];
    // of a tile: {flags | tokens << 8 (WIN: | hidden tokens' first << 16, end << 24), sequence, unit, partial state or -1: the whole unit is here}
    int4* metas = reinterpret_cast<int4*>(smem + C::OFF_META);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
    uint64_t* empty = full + C::NSTAGE;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NSTAGE; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kConsumers);
        }
        fence_mbar_init();
    }
    pdl_wait();                // the kernel before (the cache write) has completed
    pdl_launch_dependents();   // the joining kernel may start its launch beside this one
    const int B = p.block_size, logB = p.log_block, upi = p.num_kv_heads * p.nsub;
    const int tile_bytes = B * C::ROWB;
    int a, end, q = 1;          // this CTA's slots (CLUSTER: tiles of its unit), the slots of each CTA
    const int my_unit = blockIdx.x >> p.log_cluster, rank = blockIdx.x & ((1 << p.log_cluster) - 1);
    if constexpr (CLUSTER) {
        const int n = tiles_of<WIN>(p, my_unit / upi);
        a = n * rank >> p.log_cluster;
        end = n * (rank + 1) >> p.log_cluster;
        __syncthreads();                           // the barriers are visible
    } else {
        scan_slots<kThreads, WIN>(p, s_pref, s_wsum);   // and the barriers are visible
        const int total = s_pref[kThreads] * upi;
        q = quota_of(p, total, s_pref[kThreads + 1]);
        a = min(blockIdx.x * q, total);
        end = min(a + q, total);
    }

    auto produce = [&] {
        // ======================= producer warp =======================
        // Plans 32 slots at a time, one a lane, then issues their tiles.
        const uint64_t policy = l2_evict_first_policy();
        int stage = 0;
        uint32_t phase = 0;
        if (lane == 0) {
            prefetch_tensormap(&map_k);
            prefetch_tensormap(&map_v);
        }
        int4* plan = reinterpret_cast<int4*>(smem + C::OFF_PLAN);      // as metas; 0: no tile here
        int2* plan_at = reinterpret_cast<int2*>(plan + 32);            // {tile of the unit, kv head}
        int* plan_row = reinterpret_cast<int*>(plan_at + 32);          // [32][16] pool rows
        // a pool row is a whole tile of 8 or 16 tokens, or half of a tile of 32
        const int log_rt = min(logB, 4), per_block = logB - log_rt, log_rows = 7 - log_rt;
        if (!CLUSTER && lane == 0) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
        __syncwarp();
        for (int pos0 = a; pos0 < end; pos0 += 32) {
            const int pos = pos0 + lane;
            int4 m = make_int4(0, 0, 0, 0);
            int uend_of = 0;
            if (CLUSTER && pos < end) {
                const int s = my_unit / upi, u = my_unit % upi;
                m = make_int4((pos == a ? kFirst : 0) | (pos == end - 1 ? kLast : 0) |
                                  min(kFp4Tile, tokens_of<WIN>(p, s) - pos * kFp4Tile) << 8 |
                                  (WIN ? hidden_of(p, s, pos) : 0),
                              s, u, p.log_cluster ? 0 : -1);
                plan_at[lane] = make_int2(pos, u / p.nsub);
            }
            if (!CLUSTER && pos < end) {
                int s, n, base;
                locate<kThreads, WIN>(p, s_pref, upi, pos, &s, &n, &base);
                const int u = (pos - base) / n, at = (pos - base) % n, tile = at - kFp4UnitCost;
                if (tile >= 0) {
                    const int dstart = pos - tile, uend = pos - at + n;
                    uend_of = uend;
                    const int tokens = min(kFp4Tile, tokens_of<WIN>(p, s) - tile * kFp4Tile);
                    m = make_int4((tile == 0 || pos == a ? kFirst : 0) |
                                      (at == n - 1 || pos == end - 1 ? kLast : 0) | tokens << 8 |
                                      (WIN ? hidden_of(p, s, tile) : 0),
                                  s, u, dstart < a ? 0 : uend > end ? 1 : -1);
                    plan_at[lane] = make_int2(tile, u / p.nsub);
                }
            }
            plan[lane] = m;
            if (!CLUSTER && pos == end - 1 && m.x != 0 && m.w == 1)   // begun here, goes on in the next worker
                p.cuts[blockIdx.x] = make_int4(1, m.y, m.z, (uend_of - 1) / q);
            const unsigned have = __ballot_sync(0xffffffffu, m.x != 0);
            __syncwarp();                 // the plan is visible to every lane (a vote orders no memory)
            // the tiles' pool rows, 8 or 16 each (beyond the context's last block: that one's again)
#pragma unroll 4
            for (int i = lane; i < 32 << log_rows; i += 32) {
                const int l = i >> log_rows, r = i & ((1 << log_rows) - 1);
                const int4 t = plan[l];
                if (t.x == 0) continue;
                const int2 w = plan_at[l];
                const int blocks = (tile_tokens<WIN>(t.x) + B - 1) >> logB, k = min(r, (blocks << per_block) - 1);
                int at = ((w.x * kFp4Tile) >> logB) + (k >> per_block);
                if constexpr (WIN)
                    at = window_entry(window_span(min(p.context_lens[t.y], p.max_context_len), p.window, p.sinks,
                                                  logB), at);
                int blk = p.block_tables[(int64_t)t.y * p.max_blocks + at];
                if (blk < 0 || blk >= p.num_blocks) {   // block 0 in its place, as every decode here
                    set_status(p.status, PKV_DEV_BAD_BLOCK_ID);
                    blk = 0;
                }
                const int row = blk * p.num_kv_heads + w.y;
                plan_row[l * 16 + r] = per_block ? 2 * row + (k & 1) : row;
            }
            __syncwarp();
            for (unsigned left = have; left != 0; left &= left - 1) {
                const int l = __ffs(left) - 1;
                if (!mbar_wait(&empty[stage], phase ^ 1u)) {
                    set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
                    return;
                }
                if (lane == 0) {
                    const int4 t = plan[l];
                    const int kvh = plan_at[l].y, qsub = t.z - kvh * p.nsub;
                    uint8_t* sb = smem + stage * C::STAGE_BYTES;
                    // 32 or 64 tokens a gather; those past the context's last block stay out
                    const int per = 4 << log_rt, gathers = (tile_tokens<WIN>(t.x) + per - 1) >> (log_rt + 2);
                    uint32_t bytes = 2u * C::ROWB * per * gathers;
                    const uint32_t qbytes = min(HEADS, p.group - qsub * HEADS) * (HD * QT::bytes);
                    if (t.x & kFirst) bytes += qbytes;
                    metas[stage] = t;
                    mbar_arrive_expect_tx(&full[stage], bytes);
                    for (int k = 0; k < gathers; ++k) {
                        const int4 y = *reinterpret_cast<const int4*>(plan_row + l * 16 + 4 * k);
                        tma_gather4(sb + k * (per * C::ROWB), &map_k, y.x, y.y, y.z, y.w, &full[stage], policy);
                        tma_gather4(sb + C::KV_BYTES + k * (per * C::ROWB), &map_v, y.x, y.y, y.z, y.w,
                                    &full[stage], policy);
                    }
                    if (t.x & kFirst) {
                        const int64_t row = (int64_t)t.y * p.num_q_heads + kvh * p.group + qsub * HEADS;
                        bulk_g2s(sb + 2 * C::KV_BYTES,
                                 static_cast<const uint8_t*>(p.q) + row * HD * QT::bytes, qbytes,
                                 &full[stage]);
                    }
                }
                if (++stage == C::NSTAGE) { stage = 0; phase ^= 1u; }
            }
            __syncwarp();                 // the plan may be rewritten
        }
        if (!mbar_wait(&empty[stage], phase ^ 1u)) {
            set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
            return;
        }
        if (lane == 0) {
            metas[stage].x = kDone;
            mbar_arrive(&full[stage]);
        }
    };
    if (warp == kConsumers) {
        produce();
        if (CLUSTER && p.log_cluster) {
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
        return;
    }

    // ========================= consumer warps =========================
    // sequences without context: zero rows (and lengths outside the bounds are flagged once)
    {
        const int cap = p.max_context_len;
        const int64_t row = (int64_t)p.num_q_heads * HD;
        for (int s = blockIdx.x * kConsumers + warp; s < p.num_seqs; s += gridDim.x * kConsumers) {
            const int c = p.context_lens[s];
            if (lane == 0 && (c < 0 || c > cap)) set_status(p.status, PKV_DEV_BAD_CONTEXT);
            if (c <= 0 || cap == 0)              // (with CLUSTER, a unit's CTAs find nothing to join)
                for (int64_t i = lane; i < row; i += 32) store_from_float<QT>(p.out, s * row + i, 0.f);
        }
    }
    constexpr int SUB_BYTES = 64 * C::ROWB;       // from a warp's first piece of a tile to its second
    const int g = lane >> 2, c = lane & 3;
    // this lane's places in a piece: ldmatrix row (token 16 warp + 8 (mi & 1) + r of chunk
    // mi >> 1), and the scale rows of tokens g, g + 8 (K) and 2c, 2c + 8 (V)
    auto place = [&](int tok, int bytes) { return (tok >> logB) * tile_bytes + (tok & (B - 1)) * bytes; };
    const int mi = lane >> 3;
    const int two_chunks = 2 * B * 16;
    const uint32_t ld_off = place(16 * warp + 8 * (mi & 1) + (lane & 7), 16) + (mi >> 1) * B * 16;
    const int sc0 = B * (HD / 2);
    const uint32_t ks_a = sc0 + place(16 * warp + g, HD / 16), vs_a = sc0 + place(16 * warp + 2 * c, HD / 16);
    const int eight = B == 8 ? tile_bytes : 8 * (HD / 16);       // from a token's scales to token + 8's
    // byte picks: K scales of the chunks (dims 8c of each); V scales of tokens 2c, 2c + 1
    const uint32_t ksel = (c >> 1) ? 0x7531u : 0x6420u;
    const uint32_t vsel = (g >> 2) ? 0x7351u : 0x6240u;

    uint4* s_qf = reinterpret_cast<uint4*>(smem + C::OFF_QF);   // per chunk: two k-steps of (b0, b1)
    // running states of heads 8 nt + 2c ([0]) and 8 nt + 2c + 1 ([1])
    float o[NT][2 * C::NCHUNK][4];
    float m[NT][2], lift[NT][2], l[NT][2], qs[NT][2];   // lift: kLift - m
    int stage = 0;
    uint32_t phase = 0;

    // One tile: SUB pieces of 16 tokens, 64 apart, nv tokens from the first of them on, of which
    // (WIN) [ha, hb) are hidden.
    auto attend = [&](auto pieces, const uint8_t* sb, int nv, int ha, int hb) {
        constexpr int SUB = decltype(pieces)::value;
        // some of the tokens are not valid
        const bool part = nv < 64 * SUB - 48 || (WIN && ha < hb && hb > 0 && ha < 64 * SUB - 48);
        auto valid = [&](int t) { return t < nv && (!WIN || t < ha || t >= hb); };
        // ---- S^T = K Q^T ----
        float sa[SUB][NT][4];
        uint32_t da[SUB], db[SUB];     // this lane's scale byte of every chunk, rows g and g + 8
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) sa[u][nt][i] = 0.f;
            const uint8_t* sc = sb + u * SUB_BYTES + ks_a;
            if constexpr (HD == 128) {
                const uint2 ra = *reinterpret_cast<const uint2*>(sc);
                const uint2 rb = *reinterpret_cast<const uint2*>(sc + eight);
                da[u] = __byte_perm(ra.x, ra.y, ksel);
                db[u] = __byte_perm(rb.x, rb.y, ksel);
            } else {
                da[u] = __byte_perm(*reinterpret_cast<const uint32_t*>(sc), 0u, ksel);
                db[u] = __byte_perm(*reinterpret_cast<const uint32_t*>(sc + eight), 0u, ksel);
            }
        }
#pragma unroll
        for (int cp = 0; cp < C::NCHUNK / 2; ++cp) {
            uint4 qf[NT][C::NP][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int t = 0; t < C::NP; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        qf[nt][t][k] = s_qf[((nt * C::NP + t) * C::NCHUNK + 2 * cp + k) * 32 + lane];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t r[4];
                ldsm4(smem_addr(sb) + u * SUB_BYTES + ld_off + cp * two_chunks, r);
                // scales of chunks 2cp (low half) and 2cp + 1, the multiply broadcasts a half
                const uint32_t pa = cp ? e4m3x2_of<1>(da[u]) : e4m3x2_of<0>(da[u]);
                const uint32_t pb = cp ? e4m3x2_of<1>(db[u]) : e4m3x2_of<0>(db[u]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t wa = r[2 * k], wb = r[2 * k + 1];
                    const uint32_t fa = half_twice(pa, k), fb = half_twice(pb, k);
                    const uint32_t a00 = hmul2(e2m1x2_to_f16x2<0>(wa), fa), a01 = hmul2(e2m1x2_to_f16x2<0>(wb), fb);
                    const uint32_t a02 = hmul2(e2m1x2_to_f16x2<1>(wa), fa), a03 = hmul2(e2m1x2_to_f16x2<1>(wb), fb);
                    const uint32_t a10 = hmul2(e2m1x2_to_f16x2<2>(wa), fa), a11 = hmul2(e2m1x2_to_f16x2<2>(wb), fb);
                    const uint32_t a12 = hmul2(e2m1x2_to_f16x2<3>(wa), fa), a13 = hmul2(e2m1x2_to_f16x2<3>(wb), fb);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int t = 0; t < C::NP; ++t) {
                            mma_f16(sa[u][nt], a00, a01, a02, a03, qf[nt][t][k].x, qf[nt][t][k].y);
                            mma_f16(sa[u][nt], a10, a11, a12, a13, qf[nt][t][k].z, qf[nt][t][k].w);
                        }
                }
            }
        }
        // ---- running softmax: elements 0, 1 are tokens g, 2, 3 tokens g + 8, of heads 2c and
        // 2c + 1; y = logit - (running max - kLift), log2 domain ----
        uint32_t pb[SUB][NT][C::NP][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float y[SUB][4], w[SUB][4], sum[2];
            auto weights = [&] {
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[u][i] = fmaf(sa[u][nt][i], qs[nt][i & 1], lift[nt][i & 1]);
                if (part)
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!valid(g + (i & 2) * 4 + 64 * u)) y[u][i] = -INFINITY;
                sum[0] = sum[1] = 0.f;
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[u][i] = fast_exp2(y[u][i]);
                    sum[0] = u ? sum[0] + (w[u][0] + w[u][2]) : w[u][0] + w[u][2];
                    sum[1] = u ? sum[1] + (w[u][1] + w[u][3]) : w[u][1] + w[u][3];
                }
            };
            weights();
            if (__any_sync(0xffffffffu, fmaxf(sum[0], sum[1]) > kMost)) {
                float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (valid(g + (i & 2) * 4 + 64 * u)) t[i & 1] = fmaxf(t[i & 1], sa[u][nt][i] * qs[nt][i & 1]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    t[0] = fmaxf(t[0], __shfl_xor_sync(0xffffffffu, t[0], off));
                    t[1] = fmaxf(t[1], __shfl_xor_sync(0xffffffffu, t[1], off));
                }
                float r[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const bool move = t[k] > m[nt][k] + kSlack;
                    r[k] = move ? fast_exp2(m[nt][k] - t[k]) : 1.f;
                    if (move) m[nt][k] = t[k];
                    lift[nt][k] = kLift - m[nt][k];
                    l[nt][k] *= r[k];
                }
#pragma unroll
                for (int mt = 0; mt < 2 * C::NCHUNK; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[nt][mt][i] *= r[i & 1];
                weights();
            }
            l[nt][0] += sum[0];
            l[nt][1] += sum[1];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                const uint32_t ua = pack_f16(w[u][0], w[u][1]), ub = pack_f16(w[u][2], w[u][3]);
                pb[u][nt][0][0] = trans8x8(ua);
                pb[u][nt][0][1] = trans8x8(ub);
                if constexpr (C::NP == 2) {
                    pb[u][nt][1][0] = trans8x8(pack_f16_rest(w[u][0], w[u][1], ua));
                    pb[u][nt][1][1] = trans8x8(pack_f16_rest(w[u][2], w[u][3], ub));
                }
            }
        }
        // ---- O^T += V^T P^T ----
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            const uint8_t* sv = sb + C::KV_BYTES + u * SUB_BYTES;
            uint32_t va[4], vb[4];      // scale bytes: tokens 2c (words 0, 1), 2c + 1 (2, 3); + 8
            if constexpr (HD == 128) {
                const uint4 ra = *reinterpret_cast<const uint4*>(sv + vs_a);
                const uint4 rb = *reinterpret_cast<const uint4*>(sv + vs_a + eight);
                va[0] = ra.x; va[1] = ra.y; va[2] = ra.z; va[3] = ra.w;
                vb[0] = rb.x; vb[1] = rb.y; vb[2] = rb.z; vb[3] = rb.w;
            } else {
                const uint2 ra = *reinterpret_cast<const uint2*>(sv + vs_a);
                const uint2 rb = *reinterpret_cast<const uint2*>(sv + vs_a + eight);
                va[0] = ra.x; va[2] = ra.y; vb[0] = rb.x; vb[2] = rb.y;
                va[1] = va[3] = vb[1] = vb[3] = 0u;
            }
            if (part) {   // rows past the context may hold anything: scale 0 (codes are finite)
                if (!valid(64 * u + 2 * c)) va[0] = va[1] = 0u;
                if (!valid(64 * u + 2 * c + 1)) va[2] = va[3] = 0u;
                if (!valid(64 * u + 2 * c + 8)) vb[0] = vb[1] = 0u;
                if (!valid(64 * u + 2 * c + 9)) vb[2] = vb[3] = 0u;
            }
#pragma unroll
            for (int cp = 0; cp < C::NCHUNK / 2; ++cp) {
                uint32_t r[4];
                ldsm4_trans(smem_addr(sv) + ld_off + cp * two_chunks, r);
                // bytes (2c, 2c + 1) of chunk 2cp's group, then of chunk 2cp + 1's
                const uint32_t ga = __byte_perm(va[cp], va[cp + 2], vsel);
                const uint32_t gb = __byte_perm(vb[cp], vb[cp + 2], vsel);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int ch = 2 * cp + k;
                    const uint32_t wa = r[2 * k], wb = r[2 * k + 1];
                    const uint32_t fa = k ? e4m3x2_of<1>(ga) : e4m3x2_of<0>(ga);
                    const uint32_t fb = k ? e4m3x2_of<1>(gb) : e4m3x2_of<0>(gb);
                    // nibble pairs (token 2c low, 2c + 1 high) in bytes 2 and 3: dims 0, 2 and
                    // dims 1, 3 of the four.  Every nibble has its place in the product of the even
                    // (or odd) ones with two shifts at once (the multiplier's pipe has room, the
                    // logic pipe that also converts has not).
                    const uint32_t la = wa & 0x0f0f0f0fu, lb = wb & 0x0f0f0f0fu;
                    const uint32_t ea = la * p.even, eb = lb * p.even;
                    // (the odd nibbles by a mask: long documents 152 instead of 151 us; with sixteen
                    // heads 227 instead of 231)
                    const uint32_t ma = NT == 1 ? la * p.minus + wa : wa & 0xf0f0f0f0u;
                    const uint32_t mb = NT == 1 ? lb * p.minus + wb : wb & 0xf0f0f0f0u;
                    const uint32_t oa = ma * p.odd, ob = mb * p.odd;
                    const uint32_t e0 = hmul2(e2m1x2_to_f16x2<2>(ea), fa), e1 = hmul2(e2m1x2_to_f16x2<3>(ea), fa);
                    const uint32_t e2 = hmul2(e2m1x2_to_f16x2<2>(eb), fb), e3 = hmul2(e2m1x2_to_f16x2<3>(eb), fb);
                    const uint32_t d0 = hmul2(e2m1x2_to_f16x2<2>(oa), fa), d1 = hmul2(e2m1x2_to_f16x2<3>(oa), fa);
                    const uint32_t d2 = hmul2(e2m1x2_to_f16x2<2>(ob), fb), d3 = hmul2(e2m1x2_to_f16x2<3>(ob), fb);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int t = 0; t < C::NP; ++t) {
                            mma_f16(o[nt][2 * ch], e0, e1, e2, e3, pb[u][nt][t][0], pb[u][nt][t][1]);
                            mma_f16(o[nt][2 * ch + 1], d0, d1, d2, d3, pb[u][nt][t][0], pb[u][nt][t][1]);
                        }
                }
            }
        }
    };

    // CLUSTER: this CTA's state, [HEADS][HD] and (m, l) of the heads, in the ring's first stage (all of
    // the CTA's tiles have been read when it is written)
    float* mine = reinterpret_cast<float*>(smem);
    float* mine_ml = mine + HEADS * HD;
    if (CLUSTER && a == end && threadIdx.x < HEADS) {
        mine_ml[2 * threadIdx.x] = -INFINITY;
        mine_ml[2 * threadIdx.x + 1] = 0.f;
    }
    while (true) {
        if (!mbar_wait(&full[stage], phase)) {
            set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
            break;
        }
        const int4 meta = metas[stage];
        if (meta.x & kDone) break;
        const uint8_t* sb = smem + stage * C::STAGE_BYTES;
        if (meta.x & kFirst) {
            const int nh = min(HEADS, p.group - meta.z % p.nsub * HEADS);
            // q row of head 8 nt + g, scaled by a power of two into fp16 (fp16 rows as they are);
            // warp w forms the operands of chunks w, w + 4, ..: dims 32 ch + 8c .. + 7
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const bool live = 8 * nt + g < nh;
                const uint8_t* sq = sb + 2 * C::KV_BYTES + ((8 * nt + g) * HD + 8 * c) * QT::bytes;
                float up = 1.f;
                qs[nt][0] = qs[nt][1] = p.qk_scale_log2;
                if constexpr (!std::is_same<QT, F16>::value) {
                    float amax = 0.f;
#pragma unroll
                    for (int ch = 0; ch < C::NCHUNK; ++ch) {
                        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                        if (live) load8<QT>(sq + 32 * ch * QT::bytes, x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) amax = absmax_nan(x[i], amax);
                    }
                    amax = absmax_nan(__shfl_xor_sync(0xffffffffu, amax, 1), amax);
                    amax = absmax_nan(__shfl_xor_sync(0xffffffffu, amax, 2), amax);
                    const int ex = (int)(__float_as_uint(amax) >> 23) - 127;     // floor(log2), or 128
                    const int e = ex == 128 ? 0 : min(14 - ex, 126);
                    up = __uint_as_float((uint32_t)(e + 127) << 23);
                    const float back = p.qk_scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
                    qs[nt][0] = __shfl_sync(0xffffffffu, back, 8 * c);
                    qs[nt][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
                }
                for (int ch = warp; ch < C::NCHUNK; ch += kConsumers) {
                    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    if (live) load8<QT>(sq + 32 * ch * QT::bytes, x);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x0 = x[2 * i] * up, x1 = x[2 * i + 1] * up;
                        hi[i] = pack_f16(x0, x1);
                        lo[i] = C::NP == 2 ? pack_f16_rest(x0, x1, hi[i]) : 0u;
                    }
                    uint4* to = s_qf + (nt * C::NP * C::NCHUNK + ch) * 32 + lane;
                    to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if constexpr (C::NP == 2) to[C::NCHUNK * 32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
#pragma unroll
                for (int mt = 0; mt < 2 * C::NCHUNK; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[nt][mt][i] = 0.f;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    m[nt][k] = -INFINITY;
                    lift[nt][k] = INFINITY;
                    l[nt][k] = 0.f;
                }
            }
            // the operands are whole; the unit before is done with its own (it met at its end)
            named_bar_sync(1, kConsumers * 32);
        }
        const int nv = tile_tokens<WIN>(meta.x) - 16 * warp;   // tokens of the tile from this warp's first on
        const int ha = WIN ? (meta.x >> 16 & 255) - 16 * warp : 0;
        const int hb = WIN ? (int)((uint32_t)meta.x >> 24) - 16 * warp : 0;
        if constexpr (C::PIECES == 2) {
            if (nv > 64) attend(std::integral_constant<int, 2>(), sb, nv, ha, hb);
            else if (nv > 0) attend(std::integral_constant<int, 1>(), sb, nv, ha, hb);
        } else {
            for (int u = 0; u < 2; ++u)
                if (nv > 64 * u)
                    attend(std::integral_constant<int, 1>(), sb + u * SUB_BYTES, nv - 64 * u, ha - 64 * u, hb - 64 * u);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == C::NSTAGE) { stage = 0; phase ^= 1u; }
        if (!(meta.x & kLast)) continue;

        // ---------------- end of the segment: the four warps' states meet ----------------
        const int kvh = meta.z / p.nsub, qsub = meta.z % p.nsub;
        const int nh = min(HEADS, p.group - qsub * HEADS);
        float* xa = reinterpret_cast<float*>(smem + C::OFF_X);
        float* xm = xa + kConsumers * 8 * C::HS;
        float* xl = xm + kConsumers * HEADS;
        const int part = threadIdx.x & 15;                          // 16 threads a head
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], off);
                if (g == 0) {
                    xm[warp * HEADS + 8 * nt + 2 * c + k] = m[nt][k];
                    xl[warp * HEADS + 8 * nt + 2 * c + k] = l[nt][k];
                }
            }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {                           // eight heads at a time,
            if (8 * nt >= nh) break;
            const int h = 8 * nt + (threadIdx.x >> 4);
            const int64_t row = (int64_t)meta.y * p.num_q_heads + kvh * p.group + qsub * HEADS + h;
            const int64_t pi = ((int64_t)blockIdx.x * 2 + max(meta.w, 0)) * HEADS + h;
            float f[kConsumers] = {0.f};                            // the warps' shares
#pragma unroll
            for (int pass = 0; pass < HD / C::XD; ++pass) {         // 64 dims at a time
#pragma unroll
                for (int mt = 0; mt < C::XD / 16; ++mt) {
                    const int dim = 32 * (mt >> 1) + 4 * g + (mt & 1);  // [2], [3]: dim + 2
                    const float* v = o[nt][pass * (C::XD / 16) + mt];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (8 * nt + 2 * c + k < nh) {
                            float* to = xa + (warp * 8 + 2 * c + k) * C::HS + dim;
                            to[0] = v[k];
                            to[2] = v[2 + k];
                        }
                }
                named_bar_sync(1, kConsumers * 32);
                if (h < nh) {
                    if (pass == 0) {
                        float M = -INFINITY, L = 0.f;
#pragma unroll
                        for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, xm[w * HEADS + h]);
#pragma unroll
                        for (int w = 0; w < kConsumers; ++w) {
                            const float mw = xm[w * HEADS + h];
                            f[w] = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
                            L = fmaf(xl[w * HEADS + h], f[w], L);
                        }
                        if (CLUSTER && meta.w >= 0) {
                            if (part == 0) {
                                mine_ml[2 * h] = M;
                                mine_ml[2 * h + 1] = L;
                            }
                        } else if (meta.w < 0) {
                            const float inv = p.out_scale / L;
#pragma unroll
                            for (int w = 0; w < kConsumers; ++w) f[w] *= inv;
                        } else if (part == 0) {
                            p.part_ml[2 * pi] = M;
                            p.part_ml[2 * pi + 1] = L;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < C::XD / 16; ++i) {
                        const int dim = part + 16 * i;
                        float A = 0.f;
#pragma unroll
                        for (int w = 0; w < kConsumers; ++w)
                            A = fmaf(xa[(w * 8 + h - 8 * nt) * C::HS + dim], f[w], A);
                        if (CLUSTER && meta.w >= 0) mine[h * HD + pass * C::XD + dim] = A;
                        else if (meta.w < 0) store_from_float<QT>(p.out, row * HD + pass * C::XD + dim, A);
                        else p.part_acc[pi * HD + pass * C::XD + dim] = A;
                    }
                }
                named_bar_sync(1, kConsumers * 32);     // the exchange buffer is free again
            }
        }
    }
    if (CLUSTER && p.log_cluster) {
        __syncwarp();
        cluster_sync();
        // a head a warp, HD / 32 dims a lane: heads `rank`, rank + cluster, .. of the unit
        const int s = my_unit / upi, u = my_unit % upi, kvh = u / p.nsub, h0 = u % p.nsub * HEADS;
        const int nh = min(HEADS, p.group - h0), last = (1 << p.log_cluster) - 1;
        constexpr int V = HD / 32;
        if (p.context_lens[s] > 0 && p.max_context_len > 0)
            for (int h = rank + (warp << p.log_cluster); h < nh; h += kConsumers << p.log_cluster) {
                float m[kFp4Cluster], l[kFp4Cluster], A[kFp4Cluster][V], M = -INFINITY, L = 0.f, sum[V] = {0.f};
#pragma unroll
                for (int k = 0; k < kFp4Cluster; ++k) {              // every load in flight at once
                    load_from(mine_ml + 2 * h, min(k, last), m[k], l[k]);
                    load_from(mine + h * HD + V * lane, min(k, last), A[k]);
                }
#pragma unroll
                for (int k = 0; k < kFp4Cluster; ++k) M = fmaxf(M, m[k]);
#pragma unroll
                for (int k = 0; k < kFp4Cluster; ++k) {
                    if (k > last || (m[k] == -INFINITY && l[k] == 0.f)) continue;   // no tiles there
                    const float f = m[k] == -INFINITY ? 0.f : fast_exp2(m[k] - M);
                    L = fmaf(l[k], f, L);
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[i] = fmaf(A[k][i], f, sum[i]);
                }
                const int64_t row = (int64_t)s * p.num_q_heads + kvh * p.group + h0 + h;
                const float inv = p.out_scale / L;
#pragma unroll
                for (int i = 0; i < V; ++i) store_from_float<QT>(p.out, row * HD + V * lane + i, sum[i] * inv);
            }
        __syncwarp();
        cluster_sync();                 // what the others read stays until they have
    }
}

// CTA b joins the partial states of the unit that worker b began and left unfinished, if it did
// (its record in `cuts`): those of workers b, b + 1, .., in that order, and writes the unit's heads.
// The warps share the heads: warp w takes head w % nh's pieces w / nh, w / nh + warps / nh, ..., four
// pieces' loads in flight at once (heads beyond the warps come after).  A plan of its own in
// every CTA instead of the record cost 4 us a call.
template <typename QT, int HD, int NT, int THREADS>
__global__ void __launch_bounds__(THREADS) merge_fp4_kernel(DecodeFp4Params p) {
    constexpr int WARPS = THREADS / 32, V = HD / 32, FLY = 4;   // dims of a lane
    constexpr int HEADS = 8 * NT;
    __shared__ float s_acc[WARPS][HD], s_m[WARPS], s_l[WARPS];
    pdl_launch_dependents();   // the kernel after waits for this one, and this one for the decode
    pdl_wait();
    const int4 cut = __ldcg(p.cuts + blockIdx.x);
    if (cut.x == 0) return;
    const int s = cut.y, u = cut.z, w0 = blockIdx.x, w1 = cut.w;
    const int kvh = u / p.nsub, qsub = u % p.nsub;
    const int heads = min(HEADS, p.group - qsub * HEADS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int h0 = 0; h0 < heads; h0 += WARPS) {
        const int nh = min(WARPS, heads - h0);
        const int h = h0 + warp % nh, step = WARPS / nh;
        float M = -INFINITY, L = 0.f, A[V];
#pragma unroll
        for (int i = 0; i < V; ++i) A[i] = 0.f;
        if (warp / nh < step)
            for (int w = w0 + warp / nh; w <= w1; w += FLY * step) {
                float m[FLY], l[FLY], a[FLY][V], Mn = M;
#pragma unroll
                for (int k = 0; k < FLY; ++k) {
                    // a worker's state 0 is the unit it starts inside of, 1 the one it ends inside of
                    const int wk = w + k * step;
                    const int64_t pi = ((int64_t)wk * 2 + (wk == w0 ? 1 : 0)) * HEADS + h;
                    m[k] = wk <= w1 ? __ldcg(p.part_ml + 2 * pi) : -INFINITY;
                    l[k] = wk <= w1 ? __ldcg(p.part_ml + 2 * pi + 1) : 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        a[k][i] = wk <= w1 ? __ldcg(p.part_acc + pi * HD + lane + 32 * i) : 0.f;
                }
#pragma unroll
                for (int k = 0; k < FLY; ++k) Mn = fmaxf(Mn, m[k]);
                const float fo = M == -INFINITY ? 0.f : fast_exp2(M - Mn);
                L *= fo;
#pragma unroll
                for (int i = 0; i < V; ++i) A[i] *= fo;
#pragma unroll
                for (int k = 0; k < FLY; ++k) {
                    const float f = m[k] == -INFINITY ? 0.f : fast_exp2(m[k] - Mn);
                    L = fmaf(l[k], f, L);
#pragma unroll
                    for (int i = 0; i < V; ++i) A[i] = fmaf(a[k][i], f, A[i]);
                }
                M = Mn;
            }
#pragma unroll
        for (int i = 0; i < V; ++i) s_acc[warp][lane + 32 * i] = A[i];
        if (lane == 0) {
            s_m[warp] = M;
            s_l[warp] = L;
        }
        __syncthreads();
        if (warp < nh) {
            M = -INFINITY;
            for (int k = 0; k < step; ++k) M = fmaxf(M, s_m[warp + k * nh]);
            L = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) A[i] = 0.f;
            for (int k = 0; k < step; ++k) {
                const int w = warp + k * nh;
                const float f = s_m[w] == -INFINITY ? 0.f : fast_exp2(s_m[w] - M);
                L = fmaf(s_l[w], f, L);
#pragma unroll
                for (int i = 0; i < V; ++i) A[i] = fmaf(s_acc[w][lane + 32 * i], f, A[i]);
            }
            const int64_t row = (int64_t)s * p.num_q_heads + kvh * p.group + qsub * HEADS + h;
            const float inv = p.out_scale / L;
#pragma unroll
            for (int i = 0; i < V; ++i) store_from_float<QT>(p.out, row * HD + lane + 32 * i, A[i] * inv);
        }
        __syncthreads();
    }
}

template <typename QT, int HD, int NT, bool CLUSTER, bool WIN>
cudaError_t launch(const DecodeFp4Params& p0, cudaStream_t stream) {
    using C = Cfg<QT, HD, NT>;
    static int workers[64] = {0};          // CTAs the device holds at once
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    auto kernel = decode_fp4_kernel<QT, HD, NT, CLUSTER, WIN>;
    if (workers[dev] == 0) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
        if (err != cudaSuccess) return err;
        int per_sm = 0, sms = 0;
        err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, C::SMEM);
        if (err != cudaSuccess) return err;
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (err != cudaSuccess) return err;
        const int w = (per_sm > 0 ? per_sm : 1) * sms;
        workers[dev] = w < kFp4MaxWorkers / NT ? w : kFp4MaxWorkers / NT;
    }
    DecodeFp4Params p = p0;
    // pools as rows of 16 tokens of one kv head (8 in blocks of 8): what one gather moves four of
    const int rt = p.block_size < 16 ? p.block_size : 16;
    const long long pool_rows = (long long)p.num_blocks * p.num_kv_heads * (p.block_size / rt);
    CUtensorMap map_k, map_v;
    if (!encode_rows_map(&map_k, p.k_cache, rt * C::ROWB, pool_rows) ||
        !encode_rows_map(&map_v, p.v_cache, rt * C::ROWB, pool_rows))
        return cudaErrorInvalidValue;
    p.workers = workers[dev];
    p.even = 0x10010u;
    p.odd = 0x1001u;
    p.minus = ~0u;
    const int64_t units = (int64_t)p.num_seqs * p.num_kv_heads * p.nsub;
    const int grid = CLUSTER ? (int)units << p.log_cluster : p.max_workers < p.workers ? p.max_workers : p.workers;
    cudaLaunchAttribute pdl[2];
    pdl[1].id = cudaLaunchAttributeClusterDimension;
    pdl[1].val.clusterDim.x = CLUSTER ? 1 << p.log_cluster : 1;
    pdl[1].val.clusterDim.y = pdl[1].val.clusterDim.z = 1;
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    err = cudaLaunchKernelEx(&cfg, kernel, p, map_k, map_v);
    if (err != cudaSuccess || CLUSTER || grid == 1) return err;      // one worker cuts nothing
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(grid - 1), 1, 1);
    cfg.dynamicSmemBytes = 0;
    // eight warps join a unit's few states; where few units share the chip, and each leaves eight
    // states or more, sixteen do (one context of 100,000 tokens and one kv head: 22 us against 31;
    // a serving batch: 107.5 us with sixteen, 106.9 with eight)
    if (units * 8 <= grid) {
        cfg.blockDim = dim3(512, 1, 1);
        return cudaLaunchKernelEx(&cfg, merge_fp4_kernel<QT, HD, NT, 512>, p);
    }
    cfg.blockDim = dim3(256, 1, 1);
    return cudaLaunchKernelEx(&cfg, merge_fp4_kernel<QT, HD, NT, 256>, p);
}

// Clusters of 1 << log_size CTAs that the device holds at once.
template <typename QT, int HD, int NT, bool WIN>
cudaError_t resident_clusters(int log_size, int* most) {
    using C = Cfg<QT, HD, NT>;
    static int known[4][64] = {{0}};       // and one, once asked for
    int* clusters = known[log_size];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (clusters[dev] == 0) {
        auto kernel = decode_fp4_kernel<QT, HD, NT, true, WIN>;
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
        if (err != cudaSuccess) return err;
        cudaLaunchAttribute dim[1];
        dim[0].id = cudaLaunchAttributeClusterDimension;
        dim[0].val.clusterDim.x = 1 << log_size;
        dim[0].val.clusterDim.y = dim[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1 << log_size, 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = C::SMEM;
        cfg.attrs = dim;
        cfg.numAttrs = 1;
        int n = 0;
        err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (err != cudaSuccess) return err;
        clusters[dev] = n + 1;
    }
    *most = clusters[dev] - 1;
    return cudaSuccess;
}

template <typename QT, int HD, int NT, bool WIN>
cudaError_t launch_units(const DecodeFp4Params& p, cudaStream_t stream) {
    const int64_t units = (int64_t)p.num_seqs * p.num_kv_heads * p.nsub;
    const int64_t tiles = ((int64_t)p.max_seen + kFp4Tile - 1) / kFp4Tile;
    for (int log_size = tiles > 4 ? 3 : tiles > 2 ? 2 : tiles > 1; log_size >= 0; --log_size) {
        if (tiles > (log_size == 3 ? 8 : kFp4ClusterTiles) << log_size || units > kFp4MaxWorkers) continue;
        int most = 0;
        const cudaError_t err = resident_clusters<QT, HD, NT, WIN>(log_size, &most);
        if (err != cudaSuccess) return err;
        if (units > most) continue;
        DecodeFp4Params of_clusters = p;
        of_clusters.log_cluster = log_size;
        return launch<QT, HD, NT, true, WIN>(of_clusters, stream);
    }
    return launch<QT, HD, NT, false, WIN>(p, stream);
}

template <typename QT, bool WIN = false>
cudaError_t launch_decode_fp4(const DecodeFp4Params& p, cudaStream_t stream) {
    if (p.unit_heads == 16)
        return p.head_dim == 128 ? launch_units<QT, 128, 2, WIN>(p, stream) : launch_units<QT, 64, 2, WIN>(p, stream);
    return p.head_dim == 128 ? launch_units<QT, 128, 1, WIN>(p, stream) : launch_units<QT, 64, 1, WIN>(p, stream);
}

}  // namespace
}  // namespace pkv
