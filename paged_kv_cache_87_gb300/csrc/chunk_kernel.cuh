// chunk_kernel.cuh -- attention of a chunk of new tokens over a paged cache, on the tensor cores
// (tcgen05): o(p) = sum_t softmax_t(scale q.k_t) v_t over the tokens t <= p that the token at
// position p sees (all, or t > p - window and t < sinks).
//
// Organisation.  A row is a (new token, query head of the kv head's group) pair; an item is a
// sequence, a kv head and two tiles of 128 rows (TMEM lanes), which share every K/V tile of 128
// tokens.  S = Q K^T (M 128, N 128, fp32 in TMEM), a thread a row for the softmax, P over S's
// columns as 16-bit pairs, O += P V (M 128, N d).  The steps of an item are the tiles of its
// virtual context: the sinks' blocks, then the window's; what is between is neither staged nor looked up.  A
// persistent CTA an SM takes pieces (runs of steps of an item) as the planner dealt them; the ring,
// the MMAs and the softmax run on from one piece into the next.
//
// Cache types.  16 bits: TMA boxes through the block table land in the MMAs' swizzled layout.  FP8
// and 4 bits: bulk copies bring a tile's bytes into a raw ring, and four warps widen them into the
// same layout as f16, exactly (code * scale of 4 bits has 6 significant bits), kv_scale being folded
// into the logit scale and the output.  bf16 queries are scaled to f16 by a power of two per row in
// place (largest magnitude in [2^14, 2^15), undone in the row's logit scale: every bit of a value
// down to 2^-29 of the row's largest stays), since one MMA takes one operand type.  f16 weights are
// lifted 2^7 above the running maximum, so that 2^-32 of the largest still counts.
//
// Warps: 0-3 and 4-7 rows of tiles A and B; 8 takes pieces and issues loads; 9 issues the MMAs; 10
// prefetches the next Q into L2; 12-15 widen (FP8 and 4 bits only).  MMA order PV_A(j), S_A(j+1),
// PV_B(j), S_B(j+1): one tile's softmax runs under the other's products.
//
// Rows of V that no row of the item sees (past the last token, before the window, behind the
// sinks: stale, poisoned or never loaded) are zeroed in shared memory, since 0 * NaN would reach O;
// rows of K may hold anything, their scores are masked.  Every wait is bounded (2 s), and a CTA in which one
// ran out stays until its copies have landed.
//
// Measured (32 / 8 heads, d 128; us; of the products' time at 1,890 TFLOP/s): 2 x 1,024 over 15k - 31k, 4 bits 775
// (0.67); 16 x 512 over 0 - 8k, FP8 196 (0.48); 4 prompts of 4k - 16k under 1,024 + 4, bf16 823 (0.53); 1 x 37 over
// 30k, 4 bits 48 (0.20); 32 x 5 over 1k - 8k, FP8 92 (0.36 of the bytes' time).  The tile step bounds it: 3,260 cycles
// in 16 bits, 3,300 - 4,000 widened, of which the four runs of products take 2,048; Q and K both come from shared
// memory, whose 128 bytes a clock the products and the widening share.  Short items add their ends: 1,500 - 3,600
// cycles between items, 4,600 for an item's output.
#pragma once

#include <atomic>
#include <type_traits>

#include "cache_row.cuh"
#include "chunk_attention.cuh"
#include "row_math.cuh"
#include "tcgen05.cuh"
#include "tmap.cuh"

namespace pkv {
namespace {

constexpr int kT = kChunkTile;
constexpr float kSlack = 8.0f;         // log2-domain headroom before the running max moves

// NARROW: items of one row tile; its steps go to tiles A and B in turn (both hold the same rows), whose
// states the rows' threads add up at the end.  For launches with few rows a sequence: two softmaxes
// and two runs of products overlap where a lone tile's would follow each other.
template <typename QT, typename KT, int HD, bool NARROW>
struct ChunkCfg {
    static constexpr bool WIDE = !std::is_same<QT, KT>::value;      // raw bytes to be widened
    static constexpr bool FP4 = std::is_same<KT, E2M1>::value;
    using MT = typename std::conditional<WIDE, F16, QT>::type;      // operand type
    static constexpr bool SCALE_Q = WIDE && std::is_same<QT, BF16>::value;
    static constexpr int HALVES = HD / 64;                           // 128-byte column slices of a row
    static constexpr int HALF_BYTES = kT * 128;
    static constexpr int TILE_BYTES = HALVES * HALF_BYTES;           // Q tile; K or V tile as operands
    static constexpr int GROUP_HALF = 8 * 128;                       // eight tokens' slice
    static constexpr int GROUP_BYTES = HALVES * GROUP_HALF;
    static constexpr int RAW_ROW = FP4 ? HD / 2 + HD / 16 : HD;      // bytes of a cached row
    static constexpr int RAW_BYTES = kT * RAW_ROW;
    static constexpr int QTILES = NARROW ? 1 : 2;
    static constexpr int STAGES = HD == 64 ? 6 : (WIDE ? (FP4 ? 4 : 3) : 5) + NARROW;
    static constexpr int RAWS = WIDE ? (HD == 64 ? 6 : FP4 ? 3 : 4) : 0;
    static constexpr int WARPS = WIDE ? 16 : 12;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int ROW_REGS = WIDE ? 184 : 216;
    static constexpr int AUX_REGS = 72;
    static constexpr float LIFT = std::is_same<MT, F16>::value ? 7.f : 0.f;
    static constexpr int ITEM_READERS = 10 + (WIDE ? 4 : 0);
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = QTILES * TILE_BYTES;
    static constexpr int OFF_RAW = OFF_RING + STAGES * TILE_BYTES;
    static constexpr int OFF_BARS = OFF_RAW + RAWS * RAW_BYTES;
    static constexpr int NUM_BARS = 2 * STAGES + 2 * RAWS + 17;
    static constexpr int OFF_MISC = OFF_BARS + NUM_BARS * 8;         // TMEM address, abort flag
    static constexpr int OFF_ITEMS = (OFF_MISC + 8 + 15) / 16 * 16;
    static constexpr int OFF_BACK = OFF_ITEMS + 2 * 80;              // [2][256] powers of two of Q's rows
    static constexpr int OFF_ML = OFF_BACK + (SCALE_Q ? 2 * 256 : 0);  // [128] (m, l) of tile B's rows
    static constexpr int SMEM = OFF_ML + (NARROW ? kT * 8 : 0) + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
    static_assert(ROW_REGS * 256 + AUX_REGS * (THREADS - 256) <= 65536 / THREADS / 8 * 8 * THREADS,
                  "the register split fits the launch's registers");
};

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;           // S_X at 128 X (P_X over its first 64), O_X at 256 + 128 X

// ---- a piece of work, as the CTA's warps see it ----
struct ChunkItem {
    int s, kvh, q_row, q_begin;    // q_row: the first query row (token) of tile A in `query`
    int p0;                        // its position (in the virtual context, as `low` and `kv_end`)
    int qn_a, qn_b;                // tokens of tiles A and B (B may have none)
    int T_a, T_b, T;               // steps of A, of B, of the piece (NARROW: 0, 2, .. are A's, 1, 3, .. B's)
    int j0;                        // step j of the piece is tile j0 + j
    int sink_blocks, skip;         // blocks from sink_blocks on are found `skip` tokens on
    int low, kv_end;               // tokens that some row sees: [0, sinks) and [low, kv_end)
    int slot;
};
struct __align__(16) ChunkSlot {
    ChunkItem it;
    int idx;                       // -1: nothing left
    int pad[3];
};
static_assert(sizeof(ChunkSlot) == 80, "two slots fill 160 bytes");

__device__ __forceinline__ int tile_of(const ChunkItem& it, int j) {
    return it.j0 + j;
}

// What of a tile some row sees: rows [0, a) and [b, e); the rest of V is zeroed.
struct TileRows {
    int a, b, e;
    __device__ __forceinline__ bool hidden(int r) const { return r >= e || (r >= a && r < b); }
    __device__ __forceinline__ bool any() const { return e < kT || a < b; }
};
__device__ __forceinline__ TileRows rows_of_tile(const ChunkItem& it, int sinks, int t0) {
    TileRows r;
    r.a = min(max(sinks - t0, 0), kT);          // (sinks up to INT_MAX: t0 >= 0)
    r.b = min(max(it.low - t0, 0), kT);
    r.e = min(it.kv_end - t0, kT);
    return r;
}

template <bool NARROW>
__device__ __forceinline__ ChunkItem chunk_item(const ChunkParams& p, const ChunkPiece& x) {
    ChunkItem it;
    it.s = x.s;
    it.kvh = x.kvh;
    it.q_begin = x.q_begin;
    const int n = x.n, ctx = x.ctx;
    const int q0 = x.pair * (NARROW ? 1 : 2) * p.qpt;
    it.q_row = it.q_begin + q0;
    it.p0 = ctx - n + q0;
    it.qn_a = min(p.qpt, n - q0);
    it.qn_b = NARROW ? 0 : max(0, min(p.qpt, n - q0 - p.qpt));
    const ChunkSpan w = chunk_span(it.p0, it.p0 + it.qn_a + it.qn_b, p.window, p.sinks, p.log_block);
    it.low = w.low;
    it.kv_end = w.kv_end;
    it.sink_blocks = w.sink_blocks;
    it.skip = w.skip;
    it.p0 -= w.skip;
    it.j0 = x.j0;
    it.T = x.j1 - x.j0;
    it.slot = x.slot;
    if (NARROW) {
        it.T_a = (it.T + 1) / 2;
        it.T_b = it.T / 2;
        return it;
    }
    // steps of tile A alone: its last token lies in an earlier tile, perhaps
    const int steps_a = (it.p0 + it.qn_a - 1) / kT + 1;
    it.T_a = max(0, min(steps_a - x.j0, it.T));
    it.T_b = it.qn_b > 0 ? it.T : 0;
    if (it.qn_b == 0) it.T_a = it.T;
    return it;
}

// The CTA's k-th piece (index -1: none left), published in a two-slot ring.
__device__ __forceinline__ int take_item(const ChunkSlot* items, uint64_t* item_full, uint64_t* item_empty,
                                         int k, ChunkItem& it, volatile int* abort_flag, unsigned* status) {
    const int slot = k & 1;
    int idx = -1;
    if (mbar_wait(&item_full[slot], (k >> 1) & 1)) {
        idx = items[slot].idx;
        if (idx >= 0) it = items[slot].it;
    } else {
        set_status(status, PKV_DEV_WAIT_TIMEOUT);
        *abort_flag = 1;
    }
    __syncwarp(__activemask());
    if ((threadIdx.x & 31) == 0) mbar_arrive(&item_empty[slot]);
    return idx;
}

template <typename C>
struct ChunkBars {
    uint64_t *full, *empty;        // [STAGES] operands of a ring entry are there; the MMAs have read it
    uint64_t *raw_full, *raw_empty;// [RAWS] raw bytes landed; widened
    uint64_t *s_full, *p_full;     // [2] S_X computed (and PV_X before it); P_X written (128 arrivals)
    uint64_t *q_raw, *q_full;      // a piece's Q rows landed; [2] are operands (of every other piece)
    uint64_t *q_free, *drain;      // a piece's S MMAs completed; all its MMAs
    uint64_t *o_free;              // [2] O_X read by the epilogue (128 arrivals)
    uint64_t *item_full, *item_empty;   // [2]
    uint64_t* fin;                 // every MMA of the CTA completed
    uint64_t* ml;                  // NARROW: tile B's (m, l) of a piece are there (128 arrivals)
    __device__ __forceinline__ explicit ChunkBars(uint8_t* smem) {
        full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
        empty = full + C::STAGES;
        raw_full = empty + C::STAGES;
        raw_empty = raw_full + C::RAWS;
        s_full = raw_empty + C::RAWS;
        p_full = s_full + 2;
        q_raw = p_full + 2;
        q_full = q_raw + 1;
        q_free = q_full + 2;
        drain = q_free + 1;
        o_free = drain + 1;
        item_full = o_free + 2;
        item_empty = item_full + 2;
        fin = item_empty + 2;
        ml = fin + 1;
    }
};

// ---- a launch that plans for itself: the producer warp of every CTA finds its CTA's pieces ----
// As the planner (chunk_plan.cu) deals them, but for the order of the sequences, which is their own,
// and whole items, which go round the CTAs.  Called by a whole warp; lane s holds sequence s.
struct ChunkSelf {
    int q0, n, ctx, incl;              // this lane's sequence; pairs up to and including it
    int total, items, split, q;        // steps of all items; a run's
    int pos, end;                      // split: the next step of this CTA's run, its end; else the next item
    int g, base;                       // split: the pair that holds pos, its first step

    // Of pair g_ (a lane's own): its sequence, its place there, its steps (0: no such pair).
    __device__ __forceinline__ int steps_of(const ChunkParams& p, int g_, int& seq, int& pair) const {
        int l = 0;
#pragma unroll
        for (int b = 16; b; b >>= 1)
            if (__shfl_sync(0xffffffffu, incl, l + b - 1) <= g_) l += b;
        seq = l = min(l, 31);
        pair = __shfl_sync(0xffffffffu, incl, l) - 1 - g_;
        const int rows = __shfl_sync(0xffffffffu, n, l), before = __shfl_sync(0xffffffffu, ctx, l) - rows;
        if (pair < 0) return 0;
        const int a = pair * p.item_tokens, b = min(rows, a + p.item_tokens);
        return chunk_span(before + a, before + b, p.window, p.sinks, p.log_block).steps;
    }

    __device__ __forceinline__ void init(const ChunkParams& p) {
        const int lane = threadIdx.x & 31, S = p.num_seqs;
        const int64_t cap = min((int64_t)p.max_context_len, (int64_t)p.max_blocks * p.block_size);
        int walked = 0;
        bool bad = false;
        q0 = n = ctx = 0;
        if (lane < S) {
            q0 = p.query_start[lane];
            const int q1 = p.query_start[lane + 1];
            ctx = p.context_lens[lane];
            const int64_t rows = (int64_t)q1 - q0;
            if (rows >= 0 && q0 >= 0 && q1 <= p.total_q && ctx >= rows && ctx <= cap) {
                n = (int)rows;
                walked = few_tokens(p, rows, ctx);
            } else {
                bad = true;
            }
            bad |= (lane == 0 && q0 != 0) || (lane == S - 1 && q1 != p.total_q);
        }
        // sequences of few rows are another kernel's, but for those that are too long for it
        const int few = few_most(p, few_sum(walked));
        if ((int64_t)n * p.group <= p.few_rows && walked <= few) n = 0;
        incl = (n + p.item_tokens - 1) / p.item_tokens;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        int all = __shfl_sync(0xffffffffu, incl, 31);
        // (starts that run back and forth could list rows twice, and more pairs than there is room for)
        if (all > p.max_pairs) {
            bad = true;
            all = 0;
        }
        if (bad && blockIdx.x == 0) set_status(p.status, PKV_DEV_BAD_CONTEXT);
        int sum = 0, most = 0, least = INT32_MAX;
        for (int g0 = 0; g0 < all; g0 += 32) {
            int seq, pair;
            const int st = steps_of(p, g0 + lane, seq, pair);
            sum += st;
            most = max(most, st);
            if (st) least = min(least, st);
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        most = __reduce_max_sync(0xffffffffu, most);
        least = __reduce_min_sync(0xffffffffu, least);
        const int N = p.num_ctas;
        total = sum * p.num_kv_heads;
        items = all * p.num_kv_heads;
        q = max(kChunkMinRun, (total + N - 1) / N);
        split = chunk_split(total, items, most, least, N, q);
        pos = split ? min((int)blockIdx.x * q, total) : (int)blockIdx.x;
        end = split ? min(pos + q, total) : items;
        g = base = 0;
        if (split && pos < end) {
            for (int g0 = 0;; g0 += 32) {
                int seq, pair, mine = steps_of(p, g0 + lane, seq, pair) * p.num_kv_heads, x = mine;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, off);
                    if (lane >= off) x += y;
                }
                const unsigned past = __ballot_sync(0xffffffffu, base + x > pos);
                if (past) {
                    const int l = __ffs(past) - 1;
                    g = g0 + l;
                    base += __shfl_sync(0xffffffffu, x - mine, l);
                    break;
                }
                base += __shfl_sync(0xffffffffu, x, 31);
            }
        }
        if (lane == 0) p.cuts[blockIdx.x].last = -1;
    }

    __device__ __forceinline__ bool next(const ChunkParams& p, ChunkPiece& x) {
        if (pos >= end) return false;
        const int c = blockIdx.x;
        int c1 = c, st;
        x.slot = -1;
        x.j0 = 0;
        if (split) {
            while (pos >= base + (st = steps_of(p, g, x.s, x.pair)) * p.num_kv_heads) {
                base += st * p.num_kv_heads;
                ++g;
            }
            const int h = (pos - base) / st, a = base + h * st, c0 = a / q;
            c1 = (a + st - 1) / q;
            x.kvh = h;
            x.j0 = pos - a;
            x.j1 = min(st, x.j0 + end - pos);
            if (c0 != c1) x.slot = 2 * c + (c == c0);
            pos += x.j1 - x.j0;
        } else {
            g = pos / p.num_kv_heads;
            x.kvh = pos - g * p.num_kv_heads;
            x.j1 = steps_of(p, g, x.s, x.pair);
            pos += p.num_ctas;
        }
        x.q_begin = __shfl_sync(0xffffffffu, q0, x.s);
        x.n = __shfl_sync(0xffffffffu, n, x.s);
        x.ctx = __shfl_sync(0xffffffffu, ctx, x.s);
        if (x.slot == 2 * c + 1 && (threadIdx.x & 31) == 0)      // begun here, ended elsewhere
            p.cuts[c] = ChunkCut{x.kvh, x.pair, x.q_begin, x.n, c1, {0, 0, 0}};
        return true;
    }
};

// ---- the producer warp: pieces; per step the entries K_j, V_j ----
template <typename C, int HD, bool NARROW>
__device__ __forceinline__ void chunk_producer(const ChunkParams& p, const CUtensorMap* tmK,
                                               const CUtensorMap* tmV, const CUtensorMap* tmQ,
                                               uint8_t* smem, const ChunkBars<C>& b, ChunkSlot* items,
                                               volatile int* abort_flag) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        if constexpr (!C::WIDE) {
            prefetch_tensormap(tmK);
            prefetch_tensormap(tmV);
        }
        prefetch_tensormap(tmQ);
    }
    const uint64_t policy = l2_evict_last_policy();      // other items read K/V again
    const uint64_t q_policy = l2_evict_first_policy();   // a query row is read once
    const int B = p.block_size, logB = p.log_block, per_tile = kT >> logB;
    ChunkSelf self;
    ChunkPiece piece;
    ChunkHead head{};
    int next = 0, end = 0;
    if (p.self_plan) {
        self.init(p);
    } else {
        // one round of loads to the CTA's first piece
        piece = p.pieces[blockIdx.x];
        head = *p.head;
        next = p.first[blockIdx.x];
        end = head.split ? p.first[blockIdx.x + 1] : head.end;
    }
    uint64_t* ring_full = C::WIDE ? b.raw_full : b.full;
    uint64_t* ring_empty = C::WIDE ? b.raw_empty : b.empty;
    constexpr int RING = C::WIDE ? C::RAWS : C::STAGES;
    uint32_t g = 0;                                      // ring entries so far
    for (int k = 0;; ++k) {
        const int slot = k & 1;
        int idx = -1;
        if (lane == 0) {
            if (!mbar_wait(&b.item_empty[slot], ((k >> 1) & 1) ^ 1u)) {
                set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
                *abort_flag = 1;
            } else if (!*abort_flag) {
                if (p.self_plan) {
                    idx = 0;
                } else if (k == 0) {
                    idx = blockIdx.x < head.begun ? (int)blockIdx.x : -1;
                } else {
                    idx = head.split ? next++ : atomicAdd(&p.head->next, 1);
                    if (idx >= end) idx = -1;
                }
            }
        }
        idx = __shfl_sync(0xffffffffu, idx, 0);
        ChunkItem it{};
        if (idx >= 0) {
            if (p.self_plan) {
                if (!self.next(p, piece)) idx = -1;
            } else if (k > 0) {
                piece = p.pieces[idx];
            }
            if (idx >= 0) it = chunk_item<NARROW>(p, piece);
        }
        if (lane == 0) {
            items[slot].it = it;
            items[slot].idx = idx;
            mbar_arrive(&b.item_full[slot]);
        }
        if (idx < 0) break;
        // the table entries of a step, one a lane, loaded a step ahead; blocks that no row sees are
        // not looked up
        const int32_t* trow = p.block_tables + (int64_t)it.s * p.max_blocks;
        auto entry = [&](int j, unsigned& need) {
            const int t0 = tile_of(it, j) * kT, r0 = lane << logB;
            const TileRows r = rows_of_tile(it, p.sinks, t0);
            const bool in = j < it.T && lane < per_tile && r0 < r.e && (r0 < r.a || r0 + B > r.b);
            need = __ballot_sync(0xffffffffu, in);
            const int blk = (t0 >> logB) + lane;
            return in ? trow[blk < it.sink_blocks ? blk : blk + (it.skip >> logB)] : 0;
        };
        unsigned need, need_next = 0;
        int cur = entry(0, need), nxt = 0;
        bool ok = true;
        for (int i = 0; i < 2 * it.T; ++i, ++g) {
            const int j = i >> 1;
            const bool is_v = i & 1;
            if (i == 1) {
                // Q, once the previous piece's S MMAs no longer read it (behind the first K tile, so
                // that the stream begins first)
                if (lane == 0) {
                    if (k > 0 && !mbar_wait(b.q_free, (k - 1) & 1)) {
                        set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
                        *abort_flag = 1;
                    }
                    const int nx = it.qn_b > 0 ? 2 : 1;
                    uint64_t* bar = C::SCALE_Q ? b.q_raw : &b.q_full[k & 1];
                    mbar_arrive_expect_tx(bar, (uint32_t)(nx * C::HALVES * p.group * p.qpt * 128));
                    for (int X = 0; X < nx; ++X)
                        for (int h = 0; h < C::HALVES; ++h)
                            tc5::tma_load_3d(smem + C::OFF_Q + X * C::TILE_BYTES + h * C::HALF_BYTES, tmQ, 64 * h,
                                             it.kvh * p.group, it.q_row + X * p.qpt, bar, q_policy);
                }
                __syncwarp();
            }
            if (!is_v) nxt = entry(j + 1, need_next);
            const int st = (int)(g % RING);
            if (!mbar_wait(&ring_empty[st], ((g / RING) & 1) ^ 1u)) {
                set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
                *abort_flag = 1;
                ok = false;
                break;
            }
            if (lane == 0)
                mbar_arrive_expect_tx(&ring_full[st],
                                      (uint32_t)(__popc(need) << logB) * (C::WIDE ? C::RAW_ROW : HD * 2));
            __syncwarp();
            if (need >> lane & 1u) {
                int phys = cur;
                if (phys < 0 || phys >= p.num_blocks) {
                    if (!is_v) set_status(p.status, PKV_DEV_BAD_BLOCK_ID);
                    phys = 0;
                }
                if constexpr (C::WIDE) {
                    const int bytes = B * C::RAW_ROW;
                    const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                                         ((int64_t)phys * p.num_kv_heads + it.kvh) * bytes;
                    bulk_g2s_hint(smem + C::OFF_RAW + st * C::RAW_BYTES + lane * bytes, src, (uint32_t)bytes,
                                  &ring_full[st], policy);
                } else {
                    const int y = (phys * p.num_kv_heads + it.kvh) * B;
                    uint8_t* dst = smem + C::OFF_RING + st * C::TILE_BYTES + lane * B * HD * 2;
                    if constexpr (HD == 128)
                        tc5::tma_load_4d(dst, is_v ? tmV : tmK, 0, 0, 0, y >> 3, &ring_full[st], policy);
                    else
                        tma_load_2d(dst, is_v ? tmV : tmK, 0, y, &ring_full[st], policy);
                }
            }
            if (is_v) {
                cur = nxt;
                need = need_next;
            }
        }
        if (!ok) break;
    }
}

// Bits 0 .. n - 1 (none below 1, all from 32 on).
__device__ __forceinline__ uint32_t bits_below(int n) {
    uint32_t x;
    asm("shl.b32 %0, 1, %1;" : "=r"(x) : "r"(max(n, 0)));     // 0 from 32 on
    return x - 1u;
}

// ---- the widening warps (128 threads): raw entries into operands, and bf16 Q into f16 ----
// Byte of 16-byte chunk c (of the row's HD / 8) of row r in an operand tile.
template <typename C>
__device__ __forceinline__ uint32_t operand_at(int r, int c) {
    return (uint32_t)((r >> 3) * C::GROUP_BYTES + (c >> 3) * C::GROUP_HALF + (r & 7) * 128 +
                      (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// One raw entry at shared address `raw` into the operand tile at `to`, by 128 threads, in a rolled
// loop whose next loads are in flight.  Its code is short on purpose: a sub-partition runs a widening
// warp beside two softmax warps, and what does not fit its instruction cache beside them costs more
// than the loop (unrolled whole: drafts over FP8 125 us; in two copies, for rows to be zeroed and
// not: 153; with a load behind every store: 157).
template <typename C, int HD>
__device__ __forceinline__ void widen_tile(uint32_t raw, uint32_t to, int logB, int tid) {
    if constexpr (C::FP4) {
        // a thread a row: its 16 bytes of each 32 dims and the two scales of these; eight lanes read
        // 128 bytes and write eight different 16-byte columns
        const int B = 1 << logB, rr = tid & (B - 1);
        uint32_t at = raw + (tid >> logB) * (B * C::RAW_ROW) + rr * 16;
        uint32_t sc_at = raw + (tid >> logB) * (B * C::RAW_ROW) + B * (HD / 2) + rr * (HD / 16);
        uint32_t row = to + (tid >> 3) * C::GROUP_BYTES + (tid & 7) * 128, col = (tid & 7) << 4;
        uint4 w = lds128(at);
        uint16_t sc;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(sc) : "r"(sc_at) : "memory");
#pragma unroll 1
        for (int ch = 0;;) {
            uint4 w_next = w;
            uint16_t sc_next = sc;
            if (ch + 1 < HD / 32) {
                at += B * 16;
                sc_at += 2;
                w_next = lds128(at);
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(sc_next) : "r"(sc_at) : "memory");
            }
            const uint32_t pair = e4m3x2_of<0>(sc);
            const __half2 two = *reinterpret_cast<const __half2*>(&pair);
            const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 s = i < 2 ? __low2half2(two) : __high2half2(two);
                uint32_t x[4] = {e2m1x2_to_f16x2<0>(word[i]), e2m1x2_to_f16x2<1>(word[i]),
                                 e2m1x2_to_f16x2<2>(word[i]), e2m1x2_to_f16x2<3>(word[i])};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&x[e]), s);
                    x[e] = *reinterpret_cast<const uint32_t*>(&v);
                }
                sts128(row + (col ^ (i << 4)), x[0], x[1], x[2], x[3]);
            }
            if (++ch == HD / 32) break;
            col ^= 64;                                   // four columns on, in the slice's other half
            if (!(ch & 1)) row += C::GROUP_HALF;
            w = w_next;
            sc = sc_next;
        }
    } else {
        // a thread 16 codes at a time: eight lanes read 128 bytes; of a row's two halves one writes
        // its odd column first, so that eight lanes write eight different columns
        constexpr int PER = HD / 16, UNITS = kT * PER / 128;
        const int r0 = tid / PER, c = tid % PER;         // (the next unit's row is a multiple of 8 on)
        const bool odd = HD == 128 && c >= 4;
        uint32_t at = raw + tid * 16;
        uint32_t out = to + (r0 >> 3) * C::GROUP_BYTES + (r0 & 7) * 128 + (c >> 2) * C::GROUP_HALF;
        const uint32_t x7 = (r0 & 7) << 4;
        const uint32_t first = (((2 * c + odd) & 7) << 4) ^ x7, second = (((2 * c + !odd) & 7) << 4) ^ x7;
        uint4 w[2] = {lds128(at), lds128(at + 2048)};
#pragma unroll 1
        for (int u = 0;;) {
            uint4 next[2] = {w[0], w[1]};
            u += 2;
            if (u < UNITS) {
                at += 4096;
                next[0] = lds128(at);
                next[1] = lds128(at + 2048);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t a0 = odd ? w[i].z : w[i].x, a1 = odd ? w[i].w : w[i].y;
                const uint32_t b0 = odd ? w[i].x : w[i].z, b1 = odd ? w[i].y : w[i].w;
                sts128(out + first, e4m3x2_of<0>(a0), e4m3x2_of<1>(a0), e4m3x2_of<0>(a1), e4m3x2_of<1>(a1));
                sts128(out + second, e4m3x2_of<0>(b0), e4m3x2_of<1>(b0), e4m3x2_of<0>(b1), e4m3x2_of<1>(b1));
                out += 4096;                             // 128 / PER rows on: HD 128 and 64 alike
            }
            if (u >= UNITS) break;
            w[0] = next[0];
            w[1] = next[1];
        }
    }
}

// Row r of a Q tile (bf16) at shared address `tile` to f16 in place, times 2^e; returns e: `most` at
// most, so that the logit scale, times the 2^-e that undoes it, is never 0 (rows below 2^-112, or whose logits
// are nothing, lose what is 2^-24 under 2^-most).
template <typename C, int HD>
__device__ __forceinline__ int scale_q_row(uint32_t tile, int r, int most) {
    const uint32_t row = tile + r * 128, x7 = (r & 7) << 4;
    auto at = [&](int c) { return row + (c >> 3) * C::HALF_BYTES + (((c & 7) << 4) ^ x7); };
    uint32_t top = 0u;                 // the largest magnitudes of even and of odd dims
#pragma unroll 1
    for (int c0 = 0; c0 < HD / 8; c0 += 4) {
        uint4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = lds128(at(c0 + c));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            top = __vmaxu2(top, w[c].x & 0x7fff7fffu);
            top = __vmaxu2(top, w[c].y & 0x7fff7fffu);
            top = __vmaxu2(top, w[c].z & 0x7fff7fffu);
            top = __vmaxu2(top, w[c].w & 0x7fff7fffu);
        }
    }
    const int ex = (int)(max(top >> 16, top & 0xffffu) >> 7) - 127;    // floor(log2); 128: not finite
    const int e = ex == 128 ? 0 : min(14 - ex, most);
    const float up = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll 1
    for (int c0 = 0; c0 < HD / 8; c0 += 2) {
        uint4 w[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) w[c] = lds128(at(c0 + c));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 h = __floats2half2_rn(__uint_as_float(x[i] << 16) * up,
                                                    __uint_as_float(x[i] & 0xffff0000u) * up);
                x[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            sts128(at(c0 + c), x[0], x[1], x[2], x[3]);
        }
    }
    return e;
}

template <typename C, int HD>
__device__ __forceinline__ void chunk_widener(const ChunkParams& p, uint8_t* smem, const ChunkBars<C>& b,
                                              const ChunkSlot* items, volatile int* abort_flag) {
    const int tid = threadIdx.x - 384, lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(smem);
    // 2^-most times the logit scale is a normal number (of a subnormal scale, more than it)
    const int most_e = min(126, (int)(__float_as_uint(p.qk_scale_log2) >> 23) - 1);
    int st = 0, rs = 0;                                  // an entry's places, and their phases
    uint32_t st_phase = 0, rs_phase = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        ChunkItem it{};
        const int idx = take_item(items, b.item_full, b.item_empty, k, it, abort_flag, p.status);
        if (idx < 0 || *abort_flag) break;
#pragma unroll 1
        for (int i = 0; i < 2 * it.T; ++i) {
            if (!mbar_wait(&b.raw_full[rs], rs_phase) || !mbar_wait(&b.empty[st], st_phase ^ 1u)) {
                ok = false;
                break;
            }
            const uint32_t to = base + C::OFF_RING + st * C::TILE_BYTES;
            widen_tile<C, HD>(base + C::OFF_RAW + rs * C::RAW_BYTES, to, p.log_block, tid);
            if (i & 1) {
                // rows of V that no row of the item sees become zeros
                const TileRows rows = rows_of_tile(it, p.sinks, tile_of(it, i >> 1) * kT);
                if (rows.any()) {
                    named_bar_sync(2, 128);              // every row has been written
                    if (rows.hidden(tid))
#pragma unroll 1
                        for (int c = 0; c < HD / 8; ++c) sts128(to + operand_at<C>(tid, c), 0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();                    // the MMAs, and the copies that reuse the raw bytes
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&b.full[st]);
                mbar_arrive(&b.raw_empty[rs]);
            }
            if (++st == C::STAGES) { st = 0; st_phase ^= 1u; }
            if (++rs == C::RAWS) { rs = 0; rs_phase ^= 1u; }
            if (C::SCALE_Q && i == 0) {
                if (!mbar_wait(b.q_raw, k & 1)) {
                    ok = false;
                    break;
                }
                int8_t* back = reinterpret_cast<int8_t*>(smem + C::OFF_BACK) + (k & 1) * 256;
#pragma unroll 1
                for (int X = 0; X < (it.qn_b > 0 ? 2 : 1); ++X)
                    back[X * kT + tid] =
                        (int8_t)scale_q_row<C, HD>(base + C::OFF_Q + X * C::TILE_BYTES, tid, most_e);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.q_full[k & 1]);
            }
        }
    }
    if (!ok) {
        set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
        *abort_flag = 1;
    }
}

// ---- the MMA issuer (one thread) ----
template <typename C, int HD, bool NARROW>
__device__ __forceinline__ void chunk_mma(const ChunkParams& p, uint8_t* smem, uint32_t tmem,
                                          const ChunkBars<C>& b, const ChunkSlot* items,
                                          volatile int* abort_flag) {
    constexpr bool kBF16 = std::is_same<typename C::MT, BF16>::value;
    constexpr uint32_t idqk = tc5::idesc_f16(kBF16, kT, kT, false, false);
    constexpr uint32_t idpv = tc5::idesc_f16(kBF16, kT, HD, false, true);
    const uint32_t aQ = smem_addr(smem + C::OFF_Q), aR = smem_addr(smem + C::OFF_RING);
    constexpr uint32_t q_hi = tc5::desc_hi_sw128(1024), kv_hi = tc5::desc_hi_sw128(C::GROUP_BYTES);
    const uint32_t q_lo0 = tc5::desc_lo_sw128(aQ, 16), r_lo0 = tc5::desc_lo_sw128(aR, 16),
                   v_lo0 = tc5::desc_lo_sw128(aR, C::GROUP_HALF);
    auto issue_s = [&](int X, int st) {
        const uint32_t qx = q_lo0 + (uint32_t)((NARROW ? 0 : X) * (C::TILE_BYTES >> 4));
        const uint32_t kx = r_lo0 + (uint32_t)(st * (C::TILE_BYTES >> 4));
        const uint32_t d = tmem + kColS + (uint32_t)(X * kT);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
            tc5::mma_ss_w(d, qx + (uint32_t)(((k >> 2) * C::HALF_BYTES + (k & 3) * 32) >> 4), q_hi,
                          kx + (uint32_t)(((k >> 2) * C::GROUP_HALF + (k & 3) * 32) >> 4), kv_hi, idqk, k > 0);
        tc5::commit(&b.s_full[X]);
    };
    auto issue_pv = [&](int X, int st, bool acc) {
        const uint32_t vx = v_lo0 + (uint32_t)(st * (C::TILE_BYTES >> 4));
        const uint32_t d = tmem + kColO + (uint32_t)(X * kT);
        const uint32_t a = tmem + kColS + (uint32_t)(X * kT);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            tc5::mma_ts_w(d, a + (uint32_t)(8 * k), vx + (uint32_t)((k * 2 * C::GROUP_BYTES) >> 4), kv_hi, idpv,
                          acc || k > 0);
    };
    auto wait_bar = [&](uint64_t* bar, uint32_t parity) {
        const bool r = mbar_wait(bar, parity);
        tc5::fence_after_sync();
        return r;
    };
    auto wait_entry = [&](uint32_t g) { return mbar_wait(&b.full[g % C::STAGES], (g / C::STAGES) & 1); };
    bool ok = true;
    uint32_t rbase = 0, np_a = 0, np_b = 0;
    for (int k = 0; ok; ++k) {
        ChunkItem it{};
        const int idx = take_item(items, b.item_full, b.item_empty, k, it, abort_flag, p.status);
        if (idx < 0 || *abort_flag) break;
        if (!wait_bar(&b.q_full[k & 1], (k >> 1) & 1) || !wait_entry(rbase)) { ok = false; break; }
        tc5::fence_after_sync();
        if constexpr (NARROW) {
            // S_A(0), S_B(1), then PV_X(j), S_X(j + 2) of X = j & 1; one tile reads an entry
            auto score = [&](int j) {
                const uint32_t gk = rbase + 2u * j;
                if (!wait_entry(gk)) return false;
                tc5::fence_after_sync();
                issue_s(j & 1, (int)(gk % C::STAGES));
                tc5::commit(&b.empty[gk % C::STAGES]);
                if (j == it.T - 1) tc5::commit(b.q_free);
                return true;
            };
            ok = score(0) && (it.T < 2 || score(1));
            if (ok && k > 0 && (!wait_bar(&b.o_free[0], (k - 1) & 1) || !wait_bar(&b.o_free[1], (k - 1) & 1)))
                ok = false;
            for (int j = 0; j < it.T && ok; ++j) {
                const uint32_t gv = rbase + 2u * j + 1u;
                if (!wait_entry(gv) || !wait_bar(&b.p_full[j & 1], ((j & 1) ? np_b++ : np_a++) & 1)) {
                    ok = false;
                    break;
                }
                issue_pv(j & 1, (int)(gv % C::STAGES), j > 1);
                tc5::commit(&b.empty[gv % C::STAGES]);
                if (j + 2 < it.T) ok = score(j + 2);
            }
            if (!ok) break;
            tc5::commit(b.drain);
            rbase += 2u * (uint32_t)it.T;
            continue;
        }
        const int st0 = (int)(rbase % C::STAGES);
        if (it.T_a > 0) issue_s(0, st0);
        if (it.T_b > 0) issue_s(1, st0);
        tc5::commit(&b.empty[st0]);
        if (it.T == 1) tc5::commit(b.q_free);            // the piece's last S MMAs
        // the previous piece's epilogue has read O before P.V overwrites it
        if (k > 0 && (!wait_bar(&b.o_free[0], (k - 1) & 1) || !wait_bar(&b.o_free[1], (k - 1) & 1))) {
            ok = false;
            break;
        }
        for (int j = 0; j < it.T && ok; ++j) {
            const uint32_t gv = rbase + 2u * j + 1u, gk = gv + 1u;
            const int vs = (int)(gv % C::STAGES), ks = (int)(gk % C::STAGES);
            const bool next = j + 1 < it.T;
            if (!wait_entry(gv) || (next && !wait_entry(gk))) {
                ok = false;
                break;
            }
            if (j < it.T_a) {
                if (!wait_bar(&b.p_full[0], np_a++ & 1)) { ok = false; break; }
                issue_pv(0, vs, j > 0);
                if (j + 1 < it.T_a) issue_s(0, ks);
            }
            if (j < it.T_b) {
                if (!wait_bar(&b.p_full[1], np_b++ & 1)) { ok = false; break; }
                issue_pv(1, vs, j > 0);
            }
            tc5::commit(&b.empty[vs]);
            if (j + 1 < it.T_b) issue_s(1, ks);
            if (next) tc5::commit(&b.empty[ks]);
            if (j == it.T - 2) tc5::commit(b.q_free);
        }
        tc5::commit(b.drain);
        rbase += 2u * (uint32_t)it.T;
    }
    tc5::commit(b.fin);                                  // every MMA completes before the TMEM goes
    if (!mbar_wait(b.fin, 0)) ok = false;
    if (!ok) {
        set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
        *abort_flag = 1;
    }
}

template <typename QT, typename KT, int HD, bool NARROW>
__global__ void __launch_bounds__((ChunkCfg<QT, KT, HD, NARROW>::THREADS), 1) chunk_attention_kernel(
    ChunkParams p, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
    const __grid_constant__ CUtensorMap tmQ) {
    using C = ChunkCfg<QT, KT, HD, NARROW>;
    using MT = typename C::MT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const ChunkBars<C> b(smem);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    ChunkSlot* items = reinterpret_cast<ChunkSlot*>(smem + C::OFF_ITEMS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&b.full[i], C::WIDE ? 4 : 1);
            mbar_init(&b.empty[i], 1);
        }
        for (int i = 0; i < C::RAWS; ++i) {
            mbar_init(&b.raw_full[i], 1);
            mbar_init(&b.raw_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.s_full[i], 1);
            mbar_init(&b.q_full[i], C::SCALE_Q ? 4 : 1);
            mbar_init(&b.p_full[i], kT);
            mbar_init(&b.o_free[i], kT);
            mbar_init(&b.item_full[i], 1);
            mbar_init(&b.item_empty[i], C::ITEM_READERS);
        }
        mbar_init(b.q_raw, 1);
        mbar_init(b.q_free, 1);
        mbar_init(b.drain, 1);
        mbar_init(b.fin, 1);
        mbar_init(b.ml, kT);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) tc5::tmem_alloc(tmem_slot, kTmemCols);
    tc5::fence_before_sync();
    __syncthreads();
    tc5::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();   // the joining kernel waits for this one
    pdl_wait();                // the plan, and what was before it

    if (warp >= 8) {
        tc5::setmaxnreg_dec<C::AUX_REGS>();
        if (warp == 8) {
            chunk_producer<C, HD, NARROW>(p, &tmK, &tmV, &tmQ, smem, b, items, abort_flag);
        } else if (warp == 9) {
            if (lane == 0) chunk_mma<C, HD, NARROW>(p, smem, tmem, b, items, abort_flag);
            __syncwarp();
        } else if (warp == 10) {
            // a piece's Q rows into L2 when it is published, before the Q buffer frees
            for (int k = 0;; ++k) {
                ChunkItem it{};
                const int idx = take_item(items, b.item_full, b.item_empty, k, it, abort_flag, p.status);
                if (idx < 0) break;
                const int X = lane / C::HALVES;
                if (lane < 2 * C::HALVES && (X == 0 || it.qn_b > 0))
                    tc5::tma_prefetch_3d(&tmQ, 64 * (lane % C::HALVES), it.kvh * p.group, it.q_row + X * p.qpt);
            }
        } else if (C::WIDE && warp >= 12) {
            if constexpr (C::WIDE) chunk_widener<C, HD>(p, smem, b, items, abort_flag);
        }
        tc5::fence_before_sync();
        named_bar_sync(1, C::THREADS);
        if (warp == 9) {
            tc5::fence_after_sync();
            tc5::tmem_dealloc(tmem, kTmemCols);
        }
        return;
    }
    tc5::setmaxnreg_inc<C::ROW_REGS>();
    {
        // ========== rows: softmax, rescale of O, epilogue; a thread a row ==========
        const int X = warp >> 2;
        const int r = threadIdx.x & (kT - 1);
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t colS = tmem + lane_base + kColS + (uint32_t)(X * kT),
                       colO = tmem + lane_base + kColO + (uint32_t)(X * kT);
        const int G = p.group, qi = (NARROW ? 0 : X * p.qpt) + r / G;   // the row's token of the item
        const bool out32 = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        bool ok = true;
        uint32_t rbase = 0, ns = 0;
        ChunkItem it{};
        int idx = take_item(items, b.item_full, b.item_empty, 0, it, abort_flag, p.status);
        for (int k = 0; idx >= 0 && ok; ++k) {
            const int Tx = X ? it.T_b : it.T_a;
            const bool row_valid = r < (X && !NARROW ? it.qn_b : it.qn_a) * G;
            const int pos = it.p0 + qi;                     // sees t <= pos, t > pos - window or t < sinks
            float qk = p.qk_scale_log2;
            if constexpr (C::SCALE_Q) {
                // (the same slot's next phase, two pieces on, waits for this row's P: it cannot pass)
                if (Tx > 0) {
                    ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&b.q_full[k & 1], (k >> 1) & 1));
                    if (!ok) break;
                    const int e = reinterpret_cast<const int8_t*>(smem + C::OFF_BACK)[(k & 1) * 256 + (NARROW ? 0 : X * kT) + r];
                    qk *= __uint_as_float((uint32_t)(127 - e) << 23);
                }
            }
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = 0; j < Tx; ++j) {
                const bool got = !*abort_flag && mbar_wait(&b.s_full[X], ns++ & 1);
                if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                tc5::fence_after_sync();
                const int step = NARROW ? 2 * j + X : j;
                const int t0 = tile_of(it, step) * kT;
                // columns c <= lim, and of these c > low or c < kept, are seen
                const int lim = pos - t0, low = pos - p.window - t0, kept = p.sinks - t0;
                const bool masked = !__all_sync(0xffffffffu, lim >= kT - 1 && (low < 0 || kept >= kT));
                uint32_t sv[2][64];
                tc5::ld_32x32b_x64(colS, sv[0]);
                tc5::ld_32x32b_x64(colS + 64u, sv[1]);
                tc5::wait_ld();
                if (masked) {
                    // 32 columns' bits at a time (comparing each column with the three bounds became
                    // branches: 10,000 cycles a tile instead of 2,000)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t seen = bits_below(lim + 1 - 32 * w) &
                                              (~bits_below(low + 1 - 32 * w) | bits_below(kept - 32 * w));
                        if (__any_sync(0xffffffffu, seen != ~0u)) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                uint32_t& x = sv[w >> 1][32 * (w & 1) + c];
                                x = (seen >> c & 1u) ? x : __float_as_uint(-INFINITY);
                            }
                        }
                    }
                }
                float pmx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) pmx[i] = -INFINITY;
#pragma unroll
                for (int c = 0; c < kT; c += 2)
                    pmx[(c >> 1) & 3] = max3(pmx[(c >> 1) & 3], __uint_as_float(sv[c >> 6][c & 63]),
                                             __uint_as_float(sv[c >> 6][(c + 1) & 63]));
                const float mx = max3(pmx[0], pmx[1], fmaxf(pmx[2], pmx[3])) * qk;
                const float m_new = mx > m_run + kSlack ? mx : m_run;
                const bool resc = j > 0 && m_new != m_run;
                if (__any_sync(0xffffffffu, resc)) {
                    const float f = resc ? fast_exp2(m_run - m_new) : 1.f;
#pragma unroll 1
                    for (int c4 = 0; c4 < HD / 32; ++c4) {
                        uint32_t o[32];
                        tc5::ld_32x32b_x32(colO + (uint32_t)(c4 * 32), o);
                        tc5::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc5::st_32x32b_x32(colO + (uint32_t)(c4 * 32), o);
                    }
                    l_run *= f;
                }
                m_run = m_new;
                const float neg_m = m_run == -INFINITY ? 0.f : C::LIFT - m_run;
                const uint64_t scale2 = f2_pack(qk, qk), negm2 = f2_pack(neg_m, neg_m);
                uint64_t pls[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) pls[i] = 0ull;
                uint32_t pw[64];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int c = 64 * hh + 2 * e;
                        const uint64_t x = f2_fma(f2_pack(__uint_as_float(sv[c >> 6][c & 63]),
                                                          __uint_as_float(sv[c >> 6][(c + 1) & 63])),
                                                  scale2, negm2);
                        const float a = fast_exp2(f2_lo(x)), bb = fast_exp2(f2_hi(x));
                        pw[32 * hh + e] = pack2_bits<MT>(a, bb);
                        pls[e & 3] = f2_add(pls[e & 3], f2_pack(a, bb));
                    }
                }
                tc5::st_32x32b_x64(colS, pw);
                const uint64_t l2 = f2_add(f2_add(pls[0], pls[1]), f2_add(pls[2], pls[3]));
                l_run += f2_lo(l2) + f2_hi(l2);
                if constexpr (!C::WIDE) {
                    // the row tile whose P.V reads a V tile first zeroes what no row sees of it
                    const TileRows rows = rows_of_tile(it, p.sinks, t0);
                    if (rows.any() && (NARROW || X == 0 || j >= it.T_a)) {
                        const uint32_t gv = rbase + 2u * step + 1u;
                        if (!__all_sync(0xffffffffu, mbar_wait(&b.full[gv % C::STAGES], (gv / C::STAGES) & 1))) {
                            ok = false;
                            break;
                        }
                        if (rows.hidden(r)) {
                            uint8_t* vrow = smem + C::OFF_RING + (gv % C::STAGES) * C::TILE_BYTES;
#pragma unroll 1
                            for (int c = 0; c < HD / 8; ++c)
                                *reinterpret_cast<uint4*>(vrow + operand_at<C>(r, c)) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                }
                tc5::wait_st();
                tc5::fence_before_sync();
                mbar_arrive(&b.p_full[X]);
            }
            if (!ok) break;
            rbase += 2u * (uint32_t)it.T;
            ChunkItem nx{};
            idx = take_item(items, b.item_full, b.item_empty, k + 1, nx, abort_flag, p.status);
            // epilogue: every MMA of the piece has completed
            ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(b.drain, k & 1));
            if (!ok) break;
            tc5::fence_after_sync();
            if (NARROW && X == 1) {
                // tile A's threads add this state to theirs (O_B lies in the same lanes)
                reinterpret_cast<float2*>(smem + C::OFF_ML)[r] = make_float2(m_run, l_run);
                tc5::fence_before_sync();
                mbar_arrive(b.ml);
                it = nx;
                continue;
            }
            float fa = 1.f, fb = 0.f;                     // NARROW: the shares of the two states
            if constexpr (NARROW) {
                ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(b.ml, k & 1));
                if (!ok) break;
                tc5::fence_after_sync();
                if (it.T_b > 0) {
                    const float2 other = reinterpret_cast<const float2*>(smem + C::OFF_ML)[r];
                    const float M = fmaxf(m_run, other.x);
                    fa = m_run == -INFINITY ? 0.f : fast_exp2(m_run - M);
                    fb = other.x == -INFINITY ? 0.f : fast_exp2(other.x - M);
                    // (l is not 0 where its tile holds NaN but no finite score)
                    l_run = M == -INFINITY ? l_run + other.y : fmaf(l_run, fa, other.y * fb);
                    m_run = M;
                }
            }
            const bool whole = it.slot < 0;
            if (whole) {
                const float inv = l_run != 0.f ? p.out_scale / l_run : 0.f;
                fa *= inv;
                fb *= inv;
            }
            const int64_t part = (int64_t)it.slot * p.part_rows + X * kT + r;
            uint16_t* dst = static_cast<uint16_t*>(p.out) +
                            ((int64_t)(it.q_row + qi) * p.num_q_heads + it.kvh * G + r % G) * HD;
            // 32 columns at a time, in a rolled loop (code that runs once an item should not drive the
            // softmax's out of the instruction cache)
#pragma unroll 1
            for (int c4 = 0; c4 < HD / 32; ++c4) {
                uint32_t o[32];
                tc5::ld_32x32b_x32(colO + (uint32_t)(c4 * 32), o);
                tc5::wait_ld();
                if (!NARROW || it.T_b == 0) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fa);
                } else {
                    uint32_t o2[32];
                    tc5::ld_32x32b_x32(colO + (uint32_t)(kT + c4 * 32), o2);
                    tc5::wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(fmaf(__uint_as_float(o[e]), fa, __uint_as_float(o2[e]) * fb));
                }
                if (!row_valid) continue;
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = pack2_bits<QT>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                    if (out32) {
                        st_global_v8(dst + c4 * 32, o);
                        st_global_v8(dst + c4 * 32 + 16, o + 8);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<uint4*>(dst + c4 * 32)[e] =
                                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                } else if (Tx > 0) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) st_global_v8(p.part_acc + part * HD + c4 * 32 + 8 * e, o + 8 * e);
                }
            }
            if (row_valid && !whole) p.part_ml[part] = make_float2(m_run, l_run);
            tc5::fence_before_sync();
            mbar_arrive(&b.o_free[X]);
            if (NARROW) mbar_arrive(&b.o_free[1]);
            it = nx;
        }
        if (!ok) {
            set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
            *abort_flag = 1;
        }
    }
    tc5::fence_before_sync();
    named_bar_sync(1, C::THREADS);
    if (warp == 0 && *abort_flag) {
        // somebody gave up: the CTA stays until its copies have landed (a barrier that none is on its way to takes
        // the bound of a wait)
        constexpr int RING = C::WIDE ? C::RAWS : C::STAGES, QS = C::SCALE_Q ? 1 : 2;
        uint64_t* bar = lane < RING ? (C::WIDE ? b.raw_full : b.full) + lane
                                    : (C::SCALE_Q ? b.q_raw : b.q_full) + lane - RING;
        if (lane < RING + QS)
#pragma unroll 1
            for (uint32_t parity = 0; parity < 2; ++parity) (void)mbar_wait(bar, parity);
    }
}

// Joins the items that lie in several CTAs' runs, here the one that CTA blockIdx.x began and left
// unfinished, if it did: the states of CTAs c0 = blockIdx.x, c0 + 1, .. in that order, a warp a row, HD / 32 dims a lane, eight states' loads in flight.
template <typename QT, int HD>
__global__ void __launch_bounds__(256) chunk_join_kernel(ChunkParams p) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int V = HD / 32, FLY = 8;
    const ChunkCut cut = p.cuts[blockIdx.x];
    if (cut.last < 0) return;
    const int kvh = cut.kvh, c0 = blockIdx.x, c1 = cut.last, q_begin = cut.q_begin, n = cut.n, q0 = cut.pair * p.item_tokens;
    const int lane = threadIdx.x & 31, warps = gridDim.y * 8;
    for (int row = blockIdx.y * 8 + (threadIdx.x >> 5); row < p.part_rows; row += warps) {
        const int X = row >> 7, r = row & (kT - 1), tok = q0 + X * p.qpt + r / p.group;
        if (r >= p.qpt * p.group || tok >= n) continue;
        float M = -INFINITY, L = 0.f, A[V];
#pragma unroll
        for (int i = 0; i < V; ++i) A[i] = 0.f;
        for (int c = c0; c <= c1; c += FLY) {
            float m[FLY], l[FLY], a[FLY][V], Mn = M;
#pragma unroll
            for (int k = 0; k < FLY; ++k) {
                // a CTA's state 0 is of the item it starts inside of, 1 of the one it leaves
                const bool in = c + k <= c1;
                const int64_t at = (int64_t)(2 * (c + k) + (c + k == c0)) * p.part_rows + row;
                const float2 ml = in ? __ldcg(p.part_ml + at) : make_float2(-INFINITY, 0.f);
                m[k] = ml.x;
                l[k] = ml.y;
                const float* src = p.part_acc + at * HD + V * lane;
                if constexpr (V == 4) {
                    const float4 v = in ? __ldcg(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    a[k][0] = v.x; a[k][1] = v.y; a[k][2] = v.z; a[k][3] = v.w;
                } else {
                    const float2 v = in ? __ldcg(reinterpret_cast<const float2*>(src)) : make_float2(0.f, 0.f);
                    a[k][0] = v.x; a[k][1] = v.y;
                }
                Mn = fmaxf(Mn, m[k]);
            }
            if (Mn == -INFINITY) {                       // nothing seen yet (or every logit -inf)
#pragma unroll
                for (int k = 0; k < FLY; ++k) L += l[k];
                continue;
            }
            const float fo = M == -INFINITY ? 0.f : fast_exp2(M - Mn);
            L *= fo;
#pragma unroll
            for (int i = 0; i < V; ++i) A[i] *= fo;
#pragma unroll
            for (int k = 0; k < FLY; ++k) {
                if (m[k] == -INFINITY && l[k] == 0.f) continue;      // its rows of `part_acc` may be unwritten
                const float f = m[k] == -INFINITY ? 0.f : fast_exp2(m[k] - Mn);
                L = fmaf(l[k], f, L);
#pragma unroll
                for (int i = 0; i < V; ++i) A[i] = fmaf(a[k][i], f, A[i]);
            }
            M = Mn;
        }
        const float inv = L != 0.f ? p.out_scale / L : 0.f;
        const int64_t o = ((int64_t)(q_begin + tok) * p.num_q_heads + kvh * p.group + r % p.group) * HD + V * lane;
#pragma unroll
        for (int i = 0; i < V; ++i) store_from_float<QT>(p.out, o + i, A[i] * inv);
    }
}

template <typename QT, typename KT, int HD, bool NARROW>
cudaError_t launch_chunk_typed(const ChunkParams& p, cudaStream_t stream) {
    using C = ChunkCfg<QT, KT, HD, NARROW>;
    static std::atomic<bool> attr_set[64];            // (several threads may be the first)
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    auto kernel = chunk_attention_kernel<QT, KT, HD, NARROW>;
    if (!attr_set[dev]) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (err != cudaSuccess) return err;
        attr_set[dev] = true;
    }
    CUtensorMap tk{}, tv{}, tq;
    if constexpr (!C::WIDE) {
        const long long rows = (long long)p.num_blocks * p.num_kv_heads * p.block_size;
        const bool made = HD == 128 ? encode_pool_map_grouped(&tk, p.k_cache, rows, p.block_size) &&
                                          encode_pool_map_grouped(&tv, p.v_cache, rows, p.block_size)
                                    : encode_pool_map(&tk, p.k_cache, HD, 2, rows, p.block_size) &&
                                          encode_pool_map(&tv, p.v_cache, HD, 2, rows, p.block_size);
        if (!made) return cudaErrorInvalidValue;
    }
    if (!encode_chunk_q_map(&tq, p.q, p.total_q, p.num_q_heads, p.group, p.qpt, HD)) return cudaErrorInvalidValue;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.num_ctas, 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, p, tk, tv, tq);
    if (err != cudaSuccess || !p.may_split) return err;
    // eight warps a CTA, a row each at a time: few items lie in many runs each, and two rows a warp are
    // soonest through with them (one question over 4 bits 47.6 us, with four 50.6); many are cut into
    // two or three, and 2,400 CTAs with nothing to do cost 2 us
    cfg.gridDim = dim3((unsigned)p.num_ctas, (unsigned)(p.self_plan ? p.part_rows / 16 : 4), 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, chunk_join_kernel<QT, HD>, p);
}

template <typename QT, typename KT, int HD>
cudaError_t launch_chunk_rows(const ChunkParams& p, cudaStream_t stream) {
    return p.item_tokens == p.qpt ? launch_chunk_typed<QT, KT, HD, true>(p, stream)
                                  : launch_chunk_typed<QT, KT, HD, false>(p, stream);
}

template <typename QT, typename KT>
cudaError_t launch_chunk_kv(const ChunkParams& p, int head_dim, cudaStream_t stream) {
    return head_dim == 128 ? launch_chunk_rows<QT, KT, 128>(p, stream) : launch_chunk_rows<QT, KT, 64>(p, stream);
}

}  // namespace
}  // namespace pkv
