// row_tiles.cuh -- sets of eight query rows against the 64-token tiles of a paged cache, on mma.sync
// m16n8k16: what the decode under a window (decode_window_kernel.cuh) and the chunk attention of few
// rows (chunk_few_kernel.cuh) share.
//
// A CTA is a producer warp, which fills a ring of tiles, and four consumer warps, 16 tokens of every
// tile each.  Rows are the products' narrow side: S^T = K Q^T, O^T += V^T P^T, P kept in registers.  FP8
// and 4 bits are widened exactly to f16 between ldmatrix and the product, once for all sets; bf16
// queries are then scaled into f16 by a power of two per row.
#pragma once

#include "cluster.cuh"
#include "decode_mma.cuh"
#include "tmap.cuh"

namespace pkv {
namespace {

constexpr int kRowTile = 64;                  // tokens of a stage
constexpr int kRowWarps = 4;                  // consumers
constexpr int kRowThreads = 32 * (kRowWarps + 1);

// N: sets of eight rows (queries' heads) that the warps multiply with every tile; the decode's is one.
template <typename QT, typename KT, int HD, int N>
struct TileCfg {
    static constexpr bool FP8 = std::is_same<KT, E4M3>::value, FP4 = std::is_same<KT, E2M1>::value;
    using MT = typename std::conditional<FP8 || FP4, F16, QT>::type;
    static constexpr int ELEM_BYTES = FP8 || FP4 ? 1 : 2;
    static constexpr int ROWB = FP4 ? HD / 2 + HD / 16 : HD * ELEM_BYTES;
    // rows lie in slices of 128 bytes (FP8 of 64 dims: 64), under the swizzle of that width
    static constexpr int SLICE = !FP4 && ROWB == 64 ? 64 : 128;
    static constexpr int HALVES = FP4 ? 1 : ROWB / SLICE;
    static constexpr int ELEMS = SLICE / ELEM_BYTES;              // elements of a slice
    // f16 weights are taken 2^7 above the running maximum: 2^-32 of the largest still counts
    static constexpr float LIFT = std::is_same<MT, F16>::value ? 7.f : 0.f;
    static constexpr int KSTEPS = HD / 16, MTILES = HD / 16;
    static constexpr int HALF_BYTES = kRowTile * SLICE;
    static constexpr int KV_BYTES = FP4 ? kRowTile * ROWB : HALVES * HALF_BYTES;
    static constexpr int STAGE_BYTES = 2 * KV_BYTES;
    // stages of the ring: the most, and the fewest, with which a CTA more is resident (FP8, and 16 bits
    // of 128 dims).  FP8 of 64 dims, 1,340 units of 514 tokens: 26.0 us with four CTAs of six stages alone, 20.0
    // with five of five beside them, 20.9 with six of four, whose 64 registers cost 64 x 4,096 44.7 -> 47.0
    static constexpr int NSTAGE = N > 1 ? (FP4 || SLICE == 64 ? 8 : HD == 64 ? 4 : 6)
                                        : STAGE_BYTES == 32768 ? 3 : HD == 64 && STAGE_BYTES <= 8192 ? 6 : 4;
    static constexpr int FEWEST = N > 1 ? NSTAGE : SLICE == 64 ? 5 : FP8 ? 3 : STAGE_BYTES == 32768 ? 2 : NSTAGE;
    // in front of the ring: the barriers; one set: the CTA's state [8][HD], (m, l)[8]; several: the fragments
    // of Q^T, and where the rows are (their place in q and out, 64 bits, their token's in the virtual context)
    static constexpr int OFF_MINE = 128, OFF_Q = 128;
    static constexpr int OFF_ROWS = OFF_Q + N * KSTEPS * 256;
    static constexpr int OFF_RING = ((N > 1 ? OFF_ROWS + 96 * N : OFF_MINE + 8 * HD * 4 + 64) + 1023) / 1024 * 1024;
    static constexpr int smem(int stages) { return OFF_RING + stages * STAGE_BYTES + 1024; }
    static constexpr int HS = HD + 4;                             // stride of a head's row where warps meet
    static_assert(kRowWarps * 8 * N * (HS + 2) * 4 <= FEWEST * STAGE_BYTES, "the ring holds the warps' states");
    // resident, at most
    static constexpr int CTAS = N > 1                  ? (HD == 64 ? 3 : 2)
                                : STAGE_BYTES == 32768 ? 3
                                : FP4                  ? (HD == 64 ? 7 : 4)
                                : FP8                  ? (HD == 64 ? 5 : 4)
                                                       : 3;
};

// Byte offset of 16-byte chunk `chunk` of row r in a slice of a tile.
template <typename C>
__device__ __forceinline__ uint32_t tile_at(int r, int chunk) {
    return C::SLICE == 64 ? (uint32_t)(r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4)) : swz(r, chunk);
}

// Where a lane's operands of a tile are.
template <typename C, int HD>
struct TileLane {
    int warp, lane, g, c, mi;
    int rl, rv;                            // ldmatrix rows of K, and of V
    // 4 bits: this lane's ldmatrix row (token 16 warp + 8 (mi & 1) + r of chunk mi >> 1), and the scales
    // of tokens g (K) and 2c (V) of the warp's piece; 8 tokens on they are `eight` bytes on
    uint32_t ld_off, ks_at, vs_at, ksel, vsel;
    int B, eight;

    __device__ __forceinline__ TileLane(int block_size, int log_block) : B(block_size) {
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        g = lane >> 2;
        c = lane & 3;
        mi = lane >> 3;
        rl = (lane & 7) + ((lane >> 3) & 1) * 8 + 16 * warp;
        rv = (lane & 7) + (mi >> 1) * 8 + 16 * warp;
        const int tile_bytes = C::ROWB << log_block;
        auto place = [&](int tok, int bytes) { return (tok >> log_block) * tile_bytes + (tok & (B - 1)) * bytes; };
        ld_off = place(16 * warp + 8 * (mi & 1) + (lane & 7), 16) + (mi >> 1) * B * 16;
        ks_at = B * (HD / 2) + place(16 * warp + g, HD / 16);
        vs_at = B * (HD / 2) + place(16 * warp + 2 * c, HD / 16);
        eight = B == 8 ? tile_bytes : 8 * (HD / 16);
        ksel = (c >> 1) ? 0x7531u : 0x6420u;
        vsel = (g >> 2) ? 0x7351u : 0x6240u;
    }
};

// The producer warp: tiles a .. end - 1 of a context of `tokens` tokens into the ring, block j of it being
// entry(j) of the table row.
template <typename C, int HD, typename Entry>
__device__ __forceinline__ void tile_producer(const void* k_cache, const void* v_cache, const CUtensorMap* tmK,
                                              const CUtensorMap* tmV, const int32_t* trow, const Entry& entry,
                                              int tokens, int a, int end, int log_block, int num_kv_heads, int kvh,
                                              int num_blocks, int stages, uint64_t* full, uint64_t* empty,
                                              uint8_t* ring, unsigned* status) {
    const int lane = threadIdx.x & 31, logB = log_block;
    const uint64_t policy = l2_evict_first_policy();
    const int log_per = 6 - logB, blocks = (tokens - 1) >> logB;            // entries a tile; the last block
    // 32 table entries at a time, the next ones loading
    int base = a << log_per;
    auto entries = [&](int j) { return j <= blocks && j < end << log_per ? trow[entry(j)] : 0; };
    int cur = entries(base + lane), nxt = entries(base + 32 + lane);
    if (!C::FP4 && lane == 0) {
        prefetch_tensormap(tmK);
        prefetch_tensormap(tmV);
    }
    int stage = 0;
    uint32_t phase = 0;
    for (int t = a; t < end; ++t) {
        const int j0 = t << log_per, nblk = min(1 << log_per, blocks + 1 - j0);
        if (j0 >= base + 32) {
            base += 32;
            cur = nxt;
            nxt = entries(base + 32 + lane);
        }
        if (!mbar_wait(&empty[stage], phase ^ 1u)) {
            set_status(status, PKV_DEV_WAIT_TIMEOUT);
            break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], 2u * (uint32_t)(nblk << logB) * C::ROWB);
        __syncwarp();
        int phys = __shfl_sync(0xffffffffu, cur, (j0 - base + lane) & 31);
        if (lane < nblk) {
            if (phys < 0 || phys >= num_blocks) {
                set_status(status, PKV_DEV_BAD_BLOCK_ID);
                phys = 0;
            }
            uint8_t* to = ring + stage * C::STAGE_BYTES;
            if constexpr (C::FP4) {
                const int bytes = C::ROWB << logB;
                const int64_t from = ((int64_t)phys * num_kv_heads + kvh) * bytes;
                to += lane * bytes;
                bulk_g2s_hint(to, static_cast<const uint8_t*>(k_cache) + from, bytes, &full[stage], policy);
                bulk_g2s_hint(to + C::KV_BYTES, static_cast<const uint8_t*>(v_cache) + from, bytes, &full[stage],
                              policy);
            } else {
                const int y = (phys * num_kv_heads + kvh) << logB;
                to += (lane << logB) * C::SLICE;
#pragma unroll
                for (int h = 0; h < C::HALVES; ++h) {
                    tma_load_2d(to + h * C::HALF_BYTES, tmK, h * C::ELEMS, y, &full[stage], policy);
                    tma_load_2d(to + C::KV_BYTES + h * C::HALF_BYTES, tmV, h * C::ELEMS, y, &full[stage], policy);
                }
            }
        }
        if (++stage == stages) { stage = 0; phase ^= 1u; }
    }
}

// Q^T fragments of this lane's row (`live`: there is one), and the logit scales of rows 2c and 2c + 1.
template <typename C, typename QT, int HD>
__device__ __forceinline__ void tile_query(const TileLane<C, HD>& w, const uint16_t* qg, bool live,
                                           uint32_t (&qf)[C::KSTEPS][2], float& qs0, float& qs1) {
    using MT = typename C::MT;
    if constexpr (C::FP4) {
        // dims 32 ch + 8c .. + 7 of chunk ch are the pairs of k-steps 2 ch and 2 ch + 1
#pragma unroll
        for (int ch = 0; ch < HD / 32; ++ch) {
            const uint4 x = live ? reinterpret_cast<const uint4*>(qg)[4 * ch + w.c] : make_uint4(0u, 0u, 0u, 0u);
            qf[2 * ch][0] = x.x; qf[2 * ch][1] = x.y; qf[2 * ch + 1][0] = x.z; qf[2 * ch + 1][1] = x.w;
        }
    } else {
#pragma unroll
        for (int t = 0; t < C::KSTEPS; ++t) {
            const int d0 = C::FP8 ? 16 * t + 4 * w.c : 16 * t + 2 * w.c, d1 = C::FP8 ? d0 + 2 : d0 + 8;
            qf[t][0] = live ? *reinterpret_cast<const uint32_t*>(qg + d0) : 0u;
            qf[t][1] = live ? *reinterpret_cast<const uint32_t*>(qg + d1) : 0u;
        }
    }
    if constexpr (!std::is_same<QT, MT>::value) {
        // bf16 queries beside f16 operands: the row's largest magnitude to [2^14, 2^15), by 2^126 at
        // most, so that what undoes it in the logit scale is a normal number
        uint32_t top = 0u;
#pragma unroll
        for (int t = 0; t < C::KSTEPS; ++t)
            top = __vmaxu2(top, __vmaxu2(qf[t][0] & 0x7fff7fffu, qf[t][1] & 0x7fff7fffu));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = (int)(max(top >> 16, top & 0xffffu) >> 7) - 127;
        const int e = ex == 128 ? 0 : min(14 - ex, 126);
        const float up = __uint_as_float((uint32_t)(e + 127) << 23);
        const float back = qs0 * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int t = 0; t < C::KSTEPS; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __half2 x = __floats2half2_rn(__uint_as_float(qf[t][i] << 16) * up,
                                                    __uint_as_float(qf[t][i] & 0xffff0000u) * up);
                qf[t][i] = *reinterpret_cast<const uint32_t*>(&x);
            }
        qs0 = __shfl_sync(0xffffffffu, back, 8 * w.c);
        qs1 = __shfl_sync(0xffffffffu, back, 8 * w.c + 4);
    }
}

// Rows of V that are not seen may hold anything: they become zeros.
template <typename C, int HD, typename Seen>
__device__ __forceinline__ void tile_zero_rows(const TileLane<C, HD>& w, uint8_t* sb, const Seen& seen) {
    const int r = w.lane >> 1;
    if (!seen(r))
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
            for (int k = 0; k < C::SLICE / 32; ++k)
                *reinterpret_cast<uint4*>(sb + C::KV_BYTES + h * C::HALF_BYTES + (16 * w.warp + r) * C::SLICE +
                                          ((w.lane & 1) * (C::SLICE / 32) + k) * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();                        // before the ring's next copy
    __syncwarp();
}

// S^T += K Q^T of the warp's 16 tokens: elements 0, 1 of a set are token g, 2, 3 token g + 8, of rows 2c, 2c + 1.
// `q(i, k)` is set i's fragment of k-step k.  With several sets it comes from shared memory, in rolled loops:
// the fragments of three sets and their sums of O do not fit in 168 registers (which is what two CTAs an SM leave).
template <typename C, int HD, int N, typename Query>
__device__ __forceinline__ void tile_scores(const TileLane<C, HD>& w, const uint8_t* sb, const Query& q,
                                            float (&sa)[N][4]) {
    using MT = typename C::MT;
    constexpr int ROLL = N > 1 ? 2 : 8;
    const uint32_t sK = smem_addr(sb);
    if constexpr (C::FP4) {
        // a word of 8 codes of row g (g + 8) and its scale are two pairs of operands; the reduction
        // index is permuted for K and q alike
        uint32_t da, db;                         // this lane's scale byte of every chunk
        if constexpr (HD == 128) {
            const uint2 ra = *reinterpret_cast<const uint2*>(sb + w.ks_at);
            const uint2 rb = *reinterpret_cast<const uint2*>(sb + w.ks_at + w.eight);
            da = __byte_perm(ra.x, ra.y, w.ksel);
            db = __byte_perm(rb.x, rb.y, w.ksel);
        } else {
            da = __byte_perm(*reinterpret_cast<const uint32_t*>(sb + w.ks_at), 0u, w.ksel);
            db = __byte_perm(*reinterpret_cast<const uint32_t*>(sb + w.ks_at + w.eight), 0u, w.ksel);
        }
#pragma unroll ROLL
        for (int cp = 0; cp < HD / 64; ++cp) {
            uint32_t r[4];
            ldsm_x4(sK + w.ld_off + cp * 2 * w.B * 16, r);
            const uint32_t pa = cp ? e4m3x2_of<1>(da) : e4m3x2_of<0>(da);
            const uint32_t pb = cp ? e4m3x2_of<1>(db) : e4m3x2_of<0>(db);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t wa = r[2 * k], wb = r[2 * k + 1], fa = half_twice(pa, k), fb = half_twice(pb, k);
                const uint32_t x[4] = {hmul2(e2m1x2_to_f16x2<0>(wa), fa), hmul2(e2m1x2_to_f16x2<0>(wb), fb),
                                       hmul2(e2m1x2_to_f16x2<1>(wa), fa), hmul2(e2m1x2_to_f16x2<1>(wb), fb)};
                const uint32_t y[4] = {hmul2(e2m1x2_to_f16x2<2>(wa), fa), hmul2(e2m1x2_to_f16x2<2>(wb), fb),
                                       hmul2(e2m1x2_to_f16x2<3>(wa), fa), hmul2(e2m1x2_to_f16x2<3>(wb), fb)};
                const int ch = 2 * cp + k;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const uint2 q0 = q(i, 2 * ch), q1 = q(i, 2 * ch + 1);
                    Mma<MT>::run(sa[i], x, q0.x, q0.y);
                    Mma<MT>::run(sa[i], y, q1.x, q1.y);
                }
            }
        }
    } else if constexpr (C::FP8) {
#pragma unroll ROLL
        for (int pr = 0; pr < C::KSTEPS / 2; ++pr) {
            uint32_t r[4];
            ldsm_x4(sK + tile_at<C>(w.rl, 2 * pr + (w.lane >> 4)), r);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t f[4] = {e4m3x2_of<0>(r[2 * k]), e4m3x2_of<0>(r[2 * k + 1]),
                                       e4m3x2_of<1>(r[2 * k]), e4m3x2_of<1>(r[2 * k + 1])};
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const uint2 b = q(i, 2 * pr + k);
                    Mma<MT>::run(sa[i], f, b.x, b.y);
                }
            }
        }
    } else {
#pragma unroll (N > 1 ? 2 : 8)
        for (int k = 0; k < C::KSTEPS; ++k) {
            uint32_t f[4];
            ldsm_x4(sK + (k >> 2) * C::HALF_BYTES + tile_at<C>(w.rl, (k & 3) * 2 + (w.lane >> 4)), f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint2 b = q(i, k);
                Mma<MT>::run(sa[i], f, b.x, b.y);
            }
        }
    }
}

// Running softmax: x are the logits (log2) of every set, m and l of rows 2c, 2c + 1; the weights as P^T's fragments.
template <typename C, int N>
__device__ __forceinline__ void tile_softmax(const float (&x)[N][4], float (&m)[N][2], float (&l)[N][2],
                                             float (&o)[N][C::MTILES][4], uint32_t (&b)[N][2]) {
    using MT = typename C::MT;
    float mx[N][2];
    bool more = false;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mx[i][r] = fmaxf(x[i][r], x[i][r + 2]);
            more |= mx[i][r] > m[i][r] + kRescaleSlack;
        }
    // warp-wide maxima only where a lane's own passes the slack (rarely, after the first tiles)
    if (__any_sync(0xffffffffu, more)) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    mx[i][r] = fmaxf(mx[i][r], __shfl_xor_sync(0xffffffffu, mx[i][r], off));
                const bool up = mx[i][r] > m[i][r] + kRescaleSlack;
                const float f = up ? fast_exp2(m[i][r] - mx[i][r]) : 1.f;
                if (up) m[i][r] = mx[i][r];
                l[i][r] *= f;
#pragma unroll
                for (int mt = 0; mt < C::MTILES; ++mt) {
                    o[i][mt][r] *= f;
                    o[i][mt][r + 2] *= f;
                }
            }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        // (a warp that has seen nothing yet has a maximum of -inf: its weights are zeros)
        const float s0 = m[i][0] == -INFINITY ? 0.f : m[i][0] - C::LIFT, s1 = m[i][1] == -INFINITY ? 0.f : m[i][1] - C::LIFT;
        // the sum is of the weights as they are multiplied, rounded to 16 bits
        float w0, w1, w2, w3;
        const uint32_t p01 = Mma<MT>::pack(fast_exp2(x[i][0] - s0), fast_exp2(x[i][1] - s1), w0, w1);
        const uint32_t p23 = Mma<MT>::pack(fast_exp2(x[i][2] - s0), fast_exp2(x[i][3] - s1), w2, w3);
        l[i][0] += w0 + w2;
        l[i][1] += w1 + w3;
        b[i][0] = movmatrix_trans(p01);
        b[i][1] = movmatrix_trans(p23);
    }
}

// O^T += V^T P^T of the warp's 16 tokens.  (4 bits, `part`: tokens that are not seen get the scale 0.  The
// nibbles' factors `even` and `odd` are 2^4 + 2^16 and 1 + 2^12, which are arguments so that they stay products.)
template <typename C, int HD, int N, typename Seen>
__device__ __forceinline__ void tile_weigh(const TileLane<C, HD>& w, const uint8_t* sb, bool part, const Seen& seen,
                                           uint32_t even, uint32_t odd, const uint32_t (&b)[N][2],
                                           float (&o)[N][C::MTILES][4]) {
    using MT = typename C::MT;
    const uint32_t sV = smem_addr(sb) + C::KV_BYTES;
    if constexpr (C::FP4) {
        const uint8_t* sv = sb + C::KV_BYTES;
        uint32_t va[4] = {0u, 0u, 0u, 0u}, vb[4] = {0u, 0u, 0u, 0u};   // scales of tokens 2c, 2c + 1; + 8
        if constexpr (HD == 128) {
            const uint4 ra = *reinterpret_cast<const uint4*>(sv + w.vs_at);
            const uint4 rb = *reinterpret_cast<const uint4*>(sv + w.vs_at + w.eight);
            va[0] = ra.x; va[1] = ra.y; va[2] = ra.z; va[3] = ra.w;
            vb[0] = rb.x; vb[1] = rb.y; vb[2] = rb.z; vb[3] = rb.w;
        } else {
            const uint2 ra = *reinterpret_cast<const uint2*>(sv + w.vs_at);
            const uint2 rb = *reinterpret_cast<const uint2*>(sv + w.vs_at + w.eight);
            va[0] = ra.x; va[2] = ra.y; vb[0] = rb.x; vb[2] = rb.y;
        }
        if (part) {      // rows that are not seen may hold anything: scale 0 (codes are finite)
            if (!seen(2 * w.c)) va[0] = va[1] = 0u;
            if (!seen(2 * w.c + 1)) va[2] = va[3] = 0u;
            if (!seen(2 * w.c + 8)) vb[0] = vb[1] = 0u;
            if (!seen(2 * w.c + 9)) vb[2] = vb[3] = 0u;
        }
#pragma unroll
        for (int cp = 0; cp < HD / 64; ++cp) {
            uint32_t r[4];
            ldsm_x4_trans(sV + w.ld_off + cp * 2 * w.B * 16, r);
            const uint32_t ga = __byte_perm(va[cp], va[cp + 2], w.vsel), gb = __byte_perm(vb[cp], vb[cp + 2], w.vsel);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int ch = 2 * cp + k;
                const uint32_t wa = r[2 * k], wb = r[2 * k + 1];
                const uint32_t fa = k ? e4m3x2_of<1>(ga) : e4m3x2_of<0>(ga);
                const uint32_t fb = k ? e4m3x2_of<1>(gb) : e4m3x2_of<0>(gb);
                // nibble pairs (token 2c low, 2c + 1 high) in bytes 2 and 3, even dims and odd ones
                const uint32_t ea = (wa & 0x0f0f0f0fu) * even, eb = (wb & 0x0f0f0f0fu) * even;
                const uint32_t oa = (wa & 0xf0f0f0f0u) * odd, ob = (wb & 0xf0f0f0f0u) * odd;
                const uint32_t ev[4] = {hmul2(e2m1x2_to_f16x2<2>(ea), fa), hmul2(e2m1x2_to_f16x2<3>(ea), fa),
                                        hmul2(e2m1x2_to_f16x2<2>(eb), fb), hmul2(e2m1x2_to_f16x2<3>(eb), fb)};
                const uint32_t od[4] = {hmul2(e2m1x2_to_f16x2<2>(oa), fa), hmul2(e2m1x2_to_f16x2<3>(oa), fa),
                                        hmul2(e2m1x2_to_f16x2<2>(ob), fb), hmul2(e2m1x2_to_f16x2<3>(ob), fb)};
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    Mma<MT>::run(o[i][2 * ch], ev, b[i][0], b[i][1]);
                    Mma<MT>::run(o[i][2 * ch + 1], od, b[i][0], b[i][1]);
                }
            }
        }
    } else if constexpr (C::FP8) {
#pragma unroll
        for (int pr = 0; pr < C::MTILES / 2; ++pr) {
            uint32_t r[4], ev[4], od[4];
            ldsm_x4_trans(sV + tile_at<C>(w.rv, 2 * pr + (w.mi & 1)), r);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t pairs = __byte_perm(r[k], 0u, 0x3120);        // even dims' pair, odd dims'
                ev[k] = e4m3x2_of<0>(pairs);
                od[k] = e4m3x2_of<1>(pairs);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                Mma<MT>::run(o[i][2 * pr], ev, b[i][0], b[i][1]);
                Mma<MT>::run(o[i][2 * pr + 1], od, b[i][0], b[i][1]);
            }
        }
    } else {
#pragma unroll
        for (int mt = 0; mt < C::MTILES; ++mt) {
            uint32_t f[4];
            ldsm_x4_trans(sV + (mt >> 2) * C::HALF_BYTES + tile_at<C>(w.rv, (mt & 3) * 2 + (w.mi & 1)), f);
#pragma unroll
            for (int i = 0; i < N; ++i) Mma<MT>::run(o[i][mt], f, b[i][0], b[i][1]);
        }
    }
}

// The warps' states meet in the ring, which they have all read; then the CTAs' of the cluster.  `mine` is what
// the CTA offers the others (ranks 0 .. parts - 1 take part), `any`: it has seen tiles.  Row k (of `rows`) goes to
// out + place(k).
template <typename C, typename QT, int HD, int N, typename Place>
__device__ __forceinline__ void tile_finish(const TileLane<C, HD>& w, uint8_t* ring, float* mine, int rank,
                                            int parts, bool any, int rows, float out_scale, void* out,
                                            const Place& place, const float (&m)[N][2], float (&l)[N][2],
                                            const float (&o)[N][C::MTILES][4]) {
    float* mine_ml = mine + 8 * N * HD;
    named_bar_sync(1, kRowWarps * 32);                   // every tile has been read
    float* xa = reinterpret_cast<float*>(ring);          // [warp][8 N][HS]
    float* xml = xa + kRowWarps * 8 * N * C::HS;         // [warp][8 N] (m, l)
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l[i][0] += __shfl_xor_sync(0xffffffffu, l[i][0], off);
            l[i][1] += __shfl_xor_sync(0xffffffffu, l[i][1], off);
        }
        const int row = (w.warp * N + i) * 8 + 2 * w.c;
        if (w.g == 0) {
            float* to = xml + row * 2;
            to[0] = m[i][0]; to[1] = l[i][0]; to[2] = m[i][1]; to[3] = l[i][1];
        }
        if (any) {
#pragma unroll
            for (int mt = 0; mt < C::MTILES; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int dim = C::FP4   ? 32 * (mt >> 1) + 4 * w.g + (mt & 1) + 2 * (e >> 1)
                                    : C::FP8 ? 32 * (mt >> 1) + 2 * w.g + (mt & 1) + 16 * (e >> 1)
                                             : 16 * mt + w.g + 8 * (e >> 1);
                    xa[(row + (e & 1)) * C::HS + dim] = o[i][mt][e];
                }
        }
    }
    named_bar_sync(1, kRowWarps * 32);
    constexpr int V = HD / 16;                           // 16 threads a row
    const int d0 = (threadIdx.x & 15) * V;
#pragma unroll 1
    for (int h = threadIdx.x >> 4; h < 8 * N; h += 8) {
        float M = -INFINITY, L = 0.f, A[V];
#pragma unroll
        for (int i = 0; i < V; ++i) A[i] = 0.f;
        if (any) {
#pragma unroll
            for (int x = 0; x < kRowWarps; ++x) M = fmaxf(M, xml[(x * 8 * N + h) * 2]);
#pragma unroll
            for (int x = 0; x < kRowWarps; ++x) {
                const float mw = xml[(x * 8 * N + h) * 2], f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
                L = fmaf(xml[(x * 8 * N + h) * 2 + 1], f, L);
#pragma unroll
                for (int i = 0; i < V; ++i) A[i] = fmaf(xa[(x * 8 * N + h) * C::HS + d0 + i], f, A[i]);
            }
        }
        if (parts == 1) {
            const float inv = L != 0.f ? out_scale / L : 0.f;     // (a NaN stays one)
            if (h < rows)
#pragma unroll
                for (int i = 0; i < V; ++i) store_from_float<QT>(out, place(h) + d0 + i, A[i] * inv);
            continue;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) mine[h * HD + d0 + i] = A[i];
        if ((threadIdx.x & 15) == 0) {
            mine_ml[2 * h] = M;
            mine_ml[2 * h + 1] = L;
        }
    }
    if (parts == 1) return;
    __syncwarp();
    cluster_sync();
    // a row a warp, HD / 32 dims a lane: rows `rank`, rank + cluster, ..
    constexpr int W = HD / 32;
    const int last = parts - 1;
    for (int k = rank + w.warp * parts; k < rows; k += kRowWarps * parts) {
        float top = -INFINITY, sum = 0.f, acc[W] = {0.f};
#pragma unroll 1
        for (int r0 = 0; r0 < parts; r0 += 8) {
            float m8[8], l8[8], v[8][W], high = top;
#pragma unroll
            for (int r = 0; r < 8; ++r) {                // eight states' loads in flight at once
                load_from(mine_ml + 2 * k, min(r0 + r, last), m8[r], l8[r]);
                load_from(mine + k * HD + W * w.lane, min(r0 + r, last), v[r]);
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) high = fmaxf(high, m8[r]);
            const float keep = top == -INFINITY ? 0.f : fast_exp2(top - high);
            top = high;
            sum *= keep;
#pragma unroll
            for (int i = 0; i < W; ++i) acc[i] *= keep;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if (r0 + r > last || (m8[r] == -INFINITY && l8[r] == 0.f)) continue;     // no tiles there
                const float f = m8[r] == -INFINITY ? 0.f : fast_exp2(m8[r] - top);
                sum = fmaf(l8[r], f, sum);
#pragma unroll
                for (int i = 0; i < W; ++i) acc[i] = fmaf(v[r][i], f, acc[i]);
            }
        }
        const float inv = sum != 0.f ? out_scale / sum : 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) store_from_float<QT>(out, place(k) + W * w.lane + i, acc[i] * inv);
    }
    __syncwarp();
    cluster_sync();                                      // what the others read stays until they have
}

}  // namespace
}  // namespace pkv
