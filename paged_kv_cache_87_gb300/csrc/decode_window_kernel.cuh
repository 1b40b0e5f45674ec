// decode_window_kernel.cuh -- decode under a sliding window for 16-bit queries, in one launch: o = sum_t softmax_t(scale q.k_t) v_t over the tokens of the virtual context of
// window_span.cuh (the sinks' blocks, then the window's).
//
// A window bounds every unit (sequence, kv head, eight query heads), so there is nothing to plan: a
// cluster of 1, 2, 4 or 8 CTAs takes a unit, an equal run of its 64-token tiles each, and joins its
// states through distributed shared memory.  A CTA is a producer warp, which fills a ring of tiles
// (TMA boxes through the block table, 128-byte swizzle), and four consumer warps, 16 tokens of every
// tile each (five warps spread over all four sub-partitions).  Products are mma.sync m16n8k16, as in
// decode_mma.cuh: S^T = K Q^T, O^T += V^T P^T, FP8 and 4 bits widened exactly to f16 between ldmatrix and
// the product (the 4-bit tiles as decode_fp4_kernel.cuh takes them: unswizzled, by bulk copies), bf16
// queries then scaled into f16 by a power of two per head, P kept in registers.  Tokens that are hidden or past the context are masked in S and their
// rows of V zeroed in shared memory, by the warp that multiplies them.
#pragma once

#include "cluster.cuh"
#include "decode_mma.cuh"
#include "tmap.cuh"

namespace pkv {
namespace {

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The low (k = 0) or high half of an f16x2 in both halves (an operand modifier, not an operation).
__device__ __forceinline__ uint32_t half_twice(uint32_t x, int k) {
    const __half2 h = *reinterpret_cast<const __half2*>(&x);
    const __half2 t = k ? __high2half2(h) : __low2half2(h);
    return *reinterpret_cast<const uint32_t*>(&t);
}

constexpr int kWinTile = 64;                  // tokens of a stage
constexpr int kWinWarps = 4;                  // consumers
constexpr int kWinThreads = 32 * (kWinWarps + 1);

template <typename QT, typename KT, int HD>
struct WinCfg {
    static constexpr bool FP8 = std::is_same<KT, E4M3>::value, FP4 = std::is_same<KT, E2M1>::value;
    using MT = typename std::conditional<FP8 || FP4, F16, QT>::type;
    static constexpr int ELEM_BYTES = FP8 || FP4 ? 1 : 2;
    static constexpr int ROWB = FP4 ? HD / 2 + HD / 16 : HD * ELEM_BYTES;
    static constexpr int HALVES = FP4 ? 1 : ROWB / 128;
    static constexpr int ELEMS = 128 / ELEM_BYTES;                // elements of a 128-byte slice
    // f16 weights are taken 2^7 above the running maximum: 2^-32 of the largest still counts
    static constexpr float LIFT = std::is_same<MT, F16>::value ? 7.f : 0.f;
    static constexpr int KSTEPS = HD / 16, MTILES = HD / 16;
    static constexpr int HALF_BYTES = kWinTile * 128;
    static constexpr int KV_BYTES = FP4 ? kWinTile * ROWB : HALVES * HALF_BYTES;
    static constexpr int STAGE_BYTES = 2 * KV_BYTES;
    // stages of the ring: the most, and the fewest, with which a CTA more is resident (FP8)
    static constexpr int NSTAGE = STAGE_BYTES == 32768 ? 3 : FP4 && HD == 64 ? 6 : 4;
    static constexpr int FEWEST = FP8 ? 3 : STAGE_BYTES == 32768 ? 2 : NSTAGE;
    // in front of the ring: the barriers, the CTA's state [8][HD], (m, l)[8]
    static constexpr int OFF_MINE = 128;
    static constexpr int OFF_RING = (OFF_MINE + 8 * HD * 4 + 64 + 1023) / 1024 * 1024;
    static constexpr int smem(int stages) { return OFF_RING + stages * STAGE_BYTES + 1024; }
    static constexpr int HS = HD + 4;                             // stride of a head's row where warps meet
    static_assert(kWinWarps * 8 * (HS + 2) * 4 <= FEWEST * STAGE_BYTES, "the ring holds the warps' states");
    static_assert(FP4 || ROWB >= 128, "rows of 128 bytes or more");
    static constexpr int CTAS = STAGE_BYTES == 32768 ? 3 : FP4 ? (HD == 64 ? 7 : 4) : FP8 ? 4 : 3;   // resident, at most
};

template <typename QT, typename KT, int HD>
__global__ void __launch_bounds__(kWinThreads, (WinCfg<QT, KT, HD>::CTAS)) decode_window_kernel(
    DecodeParams p, int log_cluster, int stages, uint32_t even, uint32_t odd, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = WinCfg<QT, KT, HD>;
    using MT = typename C::MT;
    extern __shared__ uint8_t smem_raw[];
    // every CTA of a cluster places its state alike: the offset to the boundary is the same
    uint8_t* smem = smem_raw + (-smem_addr(smem_raw) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + C::NSTAGE;
    uint8_t* ring = smem + C::OFF_RING;
    float* mine = reinterpret_cast<float*>(smem + C::OFF_MINE);
    float* mine_ml = mine + 8 * HD;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWinWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int B = p.block_size, logB = p.log_block, upi = p.num_kv_heads * p.nsub;
    const int unit = blockIdx.x >> log_cluster, rank = blockIdx.x & ((1 << log_cluster) - 1);
    const int s = unit / upi, u = unit % upi, kvh = u / p.nsub, qsub = u % p.nsub;
    const int h0 = kvh * p.group + qsub * 8, nh = min(8, p.group - qsub * 8);
    const int64_t row0 = (int64_t)s * p.num_q_heads + h0;
    int n = p.context_lens[s];
    if (n < 0 || n > p.max_context_len) {
        if (u == 0 && rank == 0 && threadIdx.x == 0) set_status(p.status, PKV_DEV_BAD_CONTEXT);
        n = n < 0 ? 0 : p.max_context_len;
    }
    if (n == 0) {                                         // (the whole cluster leaves here)
        if (rank == 0)
            for (int i = threadIdx.x; i < nh * HD; i += kWinThreads) store_from_float<QT>(p.out, row0 * HD + i, 0.f);
        return;
    }
    const WindowSpan span = window_span(n, p.window, p.sinks, logB);
    const int tiles = (span.tokens - 1) / kWinTile + 1;
    const int a = (int)((int64_t)tiles * rank >> log_cluster), end = (int)((int64_t)tiles * (rank + 1) >> log_cluster);

    if (warp == kWinWarps) {
        // ======================= producer warp =======================
        const uint64_t policy = l2_evict_first_policy();
        const int32_t* trow = p.block_tables + (int64_t)s * p.max_blocks;
        const int log_per = 6 - logB, blocks = (span.tokens - 1) >> logB;       // entries a tile; the last block
        // 32 table entries at a time, the next ones loading
        int base = a << log_per;
        auto entries = [&](int j) { return j <= blocks && j < end << log_per ? trow[window_entry(span, j)] : 0; };
        int cur = entries(base + lane), nxt = entries(base + 32 + lane);
        if (!C::FP4 && lane == 0) {
            prefetch_tensormap(&tmK);
            prefetch_tensormap(&tmV);
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
                set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], 2u * (uint32_t)(nblk << logB) * C::ROWB);
            __syncwarp();
            int phys = __shfl_sync(0xffffffffu, cur, (j0 - base + lane) & 31);
            if (lane < nblk) {
                if (phys < 0 || phys >= p.num_blocks) {
                    set_status(p.status, PKV_DEV_BAD_BLOCK_ID);
                    phys = 0;
                }
                uint8_t* to = ring + stage * C::STAGE_BYTES;
                if constexpr (C::FP4) {
                    const int bytes = C::ROWB << logB;
                    const int64_t from = ((int64_t)phys * p.num_kv_heads + kvh) * bytes;
                    to += lane * bytes;
                    bulk_g2s_hint(to, static_cast<const uint8_t*>(p.k_cache) + from, bytes, &full[stage], policy);
                    bulk_g2s_hint(to + C::KV_BYTES, static_cast<const uint8_t*>(p.v_cache) + from, bytes, &full[stage],
                                  policy);
                } else {
                    const int y = (phys * p.num_kv_heads + kvh) << logB;
                    to += (lane << logB) * 128;
#pragma unroll
                    for (int h = 0; h < C::HALVES; ++h) {
                        tma_load_2d(to + h * C::HALF_BYTES, &tmK, h * C::ELEMS, y, &full[stage], policy);
                        tma_load_2d(to + C::KV_BYTES + h * C::HALF_BYTES, &tmV, h * C::ELEMS, y, &full[stage], policy);
                    }
                }
            }
            if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        if (log_cluster) {
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
        return;
    }

    // ========================= consumer warps =========================
    const int g = lane >> 2, c = lane & 3;
    uint32_t qf[C::KSTEPS][2];                   // Q^T fragments of head g
    float qs0 = p.qk_scale_log2, qs1 = qs0;      // logit scales of heads 2c and 2c + 1
    {
        const uint16_t* qg = static_cast<const uint16_t*>(p.q) + (row0 + g) * HD;
        const bool live = g < nh;
        if constexpr (C::FP4) {
            // dims 32 ch + 8c .. + 7 of chunk ch are the pairs of k-steps 2 ch and 2 ch + 1
#pragma unroll
            for (int ch = 0; ch < HD / 32; ++ch) {
                const uint4 w = live ? reinterpret_cast<const uint4*>(qg)[4 * ch + c] : make_uint4(0u, 0u, 0u, 0u);
                qf[2 * ch][0] = w.x; qf[2 * ch][1] = w.y; qf[2 * ch + 1][0] = w.z; qf[2 * ch + 1][1] = w.w;
            }
        } else {
#pragma unroll
            for (int t = 0; t < C::KSTEPS; ++t) {
                const int d0 = C::FP8 ? 16 * t + 4 * c : 16 * t + 2 * c, d1 = C::FP8 ? d0 + 2 : d0 + 8;
                qf[t][0] = live ? *reinterpret_cast<const uint32_t*>(qg + d0) : 0u;
                qf[t][1] = live ? *reinterpret_cast<const uint32_t*>(qg + d1) : 0u;
            }
        }
        if constexpr (!std::is_same<QT, MT>::value) {
            // bf16 queries beside f16 operands: the row's largest magnitude to [2^14, 2^15), by 2^60 at
            // most, so that what undoes it in the logit scale stays a normal number
            uint32_t top = 0u;
#pragma unroll
            for (int t = 0; t < C::KSTEPS; ++t)
                top = __vmaxu2(top, __vmaxu2(qf[t][0] & 0x7fff7fffu, qf[t][1] & 0x7fff7fffu));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = (int)(max(top >> 16, top & 0xffffu) >> 7) - 127;
            const int e = ex == 128 ? 0 : min(14 - ex, 60);
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
            qs0 = __shfl_sync(0xffffffffu, back, 8 * c);
            qs1 = __shfl_sync(0xffffffffu, back, 8 * c + 4);
        }
    }
    float o[C::MTILES][4];
#pragma unroll
    for (int mt = 0; mt < C::MTILES; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;    // of heads 2c and 2c + 1
    int stage = 0;
    uint32_t phase = 0;
    const int rl = (lane & 7) + ((lane >> 3) & 1) * 8 + 16 * warp;              // ldmatrix rows of K
    const int mi = lane >> 3, rv = (lane & 7) + (mi >> 1) * 8 + 16 * warp;      // and of V
    // 4 bits: this lane's ldmatrix row (token 16 warp + 8 (mi & 1) + r of chunk mi >> 1), and the scales
    // of tokens g (K) and 2c (V) of the warp's piece; 8 tokens on they are `eight` bytes on
    const int tile_bytes = C::ROWB << logB;
    auto place = [&](int tok, int bytes) { return (tok >> logB) * tile_bytes + (tok & (B - 1)) * bytes; };
    const uint32_t ld_off = place(16 * warp + 8 * (mi & 1) + (lane & 7), 16) + (mi >> 1) * B * 16;
    const uint32_t ks_at = B * (HD / 2) + place(16 * warp + g, HD / 16);
    const uint32_t vs_at = B * (HD / 2) + place(16 * warp + 2 * c, HD / 16);
    const int eight = B == 8 ? tile_bytes : 8 * (HD / 16);
    const uint32_t ksel = (c >> 1) ? 0x7531u : 0x6420u, vsel = (g >> 2) ? 0x7351u : 0x6240u;
    bool ok = true;
    for (int t = a; t < end; ++t) {
        if (!mbar_wait(&full[stage], phase)) {
            set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
            ok = false;
            break;
        }
        uint8_t* sb = ring + stage * C::STAGE_BYTES;
        const uint32_t sK = smem_addr(sb), sV = sK + C::KV_BYTES;
        // this warp's rows: valid ones, hidden ones
        const int t0 = t * kWinTile + 16 * warp;
        const int nv = span.tokens - t0, ha = span.hide_lo - t0, hb = span.hide_hi - t0;
        if (nv > 0) {
            auto seen = [&](int r) { return r < nv && (r < ha || r >= hb); };
            const bool part = nv < 16 || (ha < hb && ha < 16 && hb > 0);
            if (!C::FP4 && part) {
                // rows that are not seen may hold anything: V's become zeros
                const int r = lane >> 1;
                if (!seen(r))
#pragma unroll
                    for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint4*>(sb + C::KV_BYTES + h * C::HALF_BYTES + (16 * warp + r) * 128 +
                                                      ((lane & 1) * 4 + k) * 16) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();                        // before the ring's next copy
                __syncwarp();
            }
            float sa[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (C::FP4) {
                // a word of 8 codes of row g (g + 8) and its scale are two pairs of operands; the reduction
                // index is permuted for K and q alike
                uint32_t da, db;                         // this lane's scale byte of every chunk
                if constexpr (HD == 128) {
                    const uint2 ra = *reinterpret_cast<const uint2*>(sb + ks_at);
                    const uint2 rb = *reinterpret_cast<const uint2*>(sb + ks_at + eight);
                    da = __byte_perm(ra.x, ra.y, ksel);
                    db = __byte_perm(rb.x, rb.y, ksel);
                } else {
                    da = __byte_perm(*reinterpret_cast<const uint32_t*>(sb + ks_at), 0u, ksel);
                    db = __byte_perm(*reinterpret_cast<const uint32_t*>(sb + ks_at + eight), 0u, ksel);
                }
#pragma unroll
                for (int cp = 0; cp < HD / 64; ++cp) {
                    uint32_t r[4];
                    ldsm_x4(sK + ld_off + cp * 2 * B * 16, r);
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
                        Mma<MT>::run(sa, x, qf[2 * ch][0], qf[2 * ch][1]);
                        Mma<MT>::run(sa, y, qf[2 * ch + 1][0], qf[2 * ch + 1][1]);
                    }
                }
            } else if constexpr (C::FP8) {
#pragma unroll
                for (int pr = 0; pr < C::KSTEPS / 2; ++pr) {
                    uint32_t r[4];
                    ldsm_x4(sK + swz(rl, 2 * pr + (lane >> 4)), r);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t f[4] = {e4m3x2_of<0>(r[2 * k]), e4m3x2_of<0>(r[2 * k + 1]),
                                               e4m3x2_of<1>(r[2 * k]), e4m3x2_of<1>(r[2 * k + 1])};
                        Mma<MT>::run(sa, f, qf[2 * pr + k][0], qf[2 * pr + k][1]);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < C::KSTEPS; ++k) {
                    uint32_t f[4];
                    ldsm_x4(sK + (k >> 2) * C::HALF_BYTES + swz(rl, (k & 3) * 2 + (lane >> 4)), f);
                    Mma<MT>::run(sa, f, qf[k][0], qf[k][1]);
                }
            }
            // running softmax: elements 0, 1 are token g, 2, 3 token g + 8, of heads 2c and 2c + 1
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = sa[e] * (e & 1 ? qs1 : qs0);
            if (part) {
                if (!seen(g)) x[0] = x[1] = -INFINITY;
                if (!seen(g + 8)) x[2] = x[3] = -INFINITY;
            }
            float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
            // a warp-wide maximum only where a lane's own passes the slack (rarely, after the first tiles)
            if (__any_sync(0xffffffffu, mx0 > m0 + kRescaleSlack || mx1 > m1 + kRescaleSlack)) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
                }
                const bool n0 = mx0 > m0 + kRescaleSlack, n1 = mx1 > m1 + kRescaleSlack;
                const float r0 = n0 ? fast_exp2(m0 - mx0) : 1.f, r1 = n1 ? fast_exp2(m1 - mx1) : 1.f;
                if (n0) m0 = mx0;
                if (n1) m1 = mx1;
                l0 *= r0;
                l1 *= r1;
#pragma unroll
                for (int mt = 0; mt < C::MTILES; ++mt) {
                    o[mt][0] *= r0;
                    o[mt][2] *= r0;
                    o[mt][1] *= r1;
                    o[mt][3] *= r1;
                }
            }
            // (a warp that has seen nothing yet has a maximum of -inf: its weights are zeros)
            const float s0 = m0 == -INFINITY ? 0.f : m0 - C::LIFT, s1 = m1 == -INFINITY ? 0.f : m1 - C::LIFT;
            const float w0 = fast_exp2(x[0] - s0), w1 = fast_exp2(x[1] - s1), w2 = fast_exp2(x[2] - s0),
                        w3 = fast_exp2(x[3] - s1);
            float unused;
            const uint32_t p01 = Mma<MT>::pack(w0, w1, unused, unused), p23 = Mma<MT>::pack(w2, w3, unused, unused);
            l0 += w0 + w2;
            l1 += w1 + w3;
            const uint32_t b0 = movmatrix_trans(p01), b1 = movmatrix_trans(p23);
            if constexpr (C::FP4) {
                const uint8_t* sv = sb + C::KV_BYTES;
                uint32_t va[4] = {0u, 0u, 0u, 0u}, vb[4] = {0u, 0u, 0u, 0u};   // scales of tokens 2c, 2c + 1; + 8
                if constexpr (HD == 128) {
                    const uint4 ra = *reinterpret_cast<const uint4*>(sv + vs_at);
                    const uint4 rb = *reinterpret_cast<const uint4*>(sv + vs_at + eight);
                    va[0] = ra.x; va[1] = ra.y; va[2] = ra.z; va[3] = ra.w;
                    vb[0] = rb.x; vb[1] = rb.y; vb[2] = rb.z; vb[3] = rb.w;
                } else {
                    const uint2 ra = *reinterpret_cast<const uint2*>(sv + vs_at);
                    const uint2 rb = *reinterpret_cast<const uint2*>(sv + vs_at + eight);
                    va[0] = ra.x; va[2] = ra.y; vb[0] = rb.x; vb[2] = rb.y;
                }
                if (part) {      // rows that are not seen may hold anything: scale 0 (codes are finite)
                    if (!seen(2 * c)) va[0] = va[1] = 0u;
                    if (!seen(2 * c + 1)) va[2] = va[3] = 0u;
                    if (!seen(2 * c + 8)) vb[0] = vb[1] = 0u;
                    if (!seen(2 * c + 9)) vb[2] = vb[3] = 0u;
                }
#pragma unroll
                for (int cp = 0; cp < HD / 64; ++cp) {
                    uint32_t r[4];
                    ldsm_x4_trans(sV + ld_off + cp * 2 * B * 16, r);
                    const uint32_t ga = __byte_perm(va[cp], va[cp + 2], vsel), gb = __byte_perm(vb[cp], vb[cp + 2], vsel);
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
                        Mma<MT>::run(o[2 * ch], ev, b0, b1);
                        Mma<MT>::run(o[2 * ch + 1], od, b0, b1);
                    }
                }
            } else if constexpr (C::FP8) {
#pragma unroll
                for (int pr = 0; pr < C::MTILES / 2; ++pr) {
                    uint32_t r[4], ev[4], od[4];
                    ldsm_x4_trans(sV + swz(rv, 2 * pr + (mi & 1)), r);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t w = __byte_perm(r[k], 0u, 0x3120);        // even dims' pair, odd dims'
                        ev[k] = e4m3x2_of<0>(w);
                        od[k] = e4m3x2_of<1>(w);
                    }
                    Mma<MT>::run(o[2 * pr], ev, b0, b1);
                    Mma<MT>::run(o[2 * pr + 1], od, b0, b1);
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < C::MTILES; ++mt) {
                    uint32_t f[4];
                    ldsm_x4_trans(sV + (mt >> 2) * C::HALF_BYTES + swz(rv, (mt & 3) * 2 + (mi & 1)), f);
                    Mma<MT>::run(o[mt], f, b0, b1);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
    }

    // ---------------- the four warps' states meet, in the ring ----------------
    named_bar_sync(1, kWinWarps * 32);                   // every tile has been read
    float* xa = reinterpret_cast<float*>(ring);          // [warp][8][HS]
    float* xml = xa + kWinWarps * 8 * C::HS;             // [warp][8] (m, l)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, off);
        l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if (g == 0) {
        float* to = xml + (warp * 8 + 2 * c) * 2;
        to[0] = m0; to[1] = l0; to[2] = m1; to[3] = l1;
    }
    if (a < end) {
#pragma unroll
        for (int mt = 0; mt < C::MTILES; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dim = C::FP4   ? 32 * (mt >> 1) + 4 * g + (mt & 1) + 2 * (e >> 1)
                                : C::FP8 ? 32 * (mt >> 1) + 2 * g + (mt & 1) + 16 * (e >> 1)
                                         : 16 * mt + g + 8 * (e >> 1);
                xa[(warp * 8 + 2 * c + (e & 1)) * C::HS + dim] = o[mt][e];
            }
    }
    named_bar_sync(1, kWinWarps * 32);
    constexpr int V = HD / 16;                           // 16 threads a head
    const int h = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * V;
    float M = -INFINITY, L = 0.f, A[V];
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = 0.f;
    if (a < end && ok) {
#pragma unroll
        for (int w = 0; w < kWinWarps; ++w) M = fmaxf(M, xml[(w * 8 + h) * 2]);
#pragma unroll
        for (int w = 0; w < kWinWarps; ++w) {
            const float mw = xml[(w * 8 + h) * 2], f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
            L = fmaf(xml[(w * 8 + h) * 2 + 1], f, L);
#pragma unroll
            for (int i = 0; i < V; ++i) A[i] = fmaf(xa[(w * 8 + h) * C::HS + d0 + i], f, A[i]);
        }
    }
    if (log_cluster == 0) {
        const float inv = L != 0.f ? p.out_scale / L : 0.f;   // (a NaN stays one)
        if (h < nh)
#pragma unroll
            for (int i = 0; i < V; ++i) store_from_float<QT>(p.out, (row0 + h) * HD + d0 + i, A[i] * inv);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) mine[h * HD + d0 + i] = A[i];
    if ((threadIdx.x & 15) == 0) {
        mine_ml[2 * h] = M;
        mine_ml[2 * h + 1] = L;
    }
    cluster_sync();
    // a head a warp, HD / 32 dims a lane: heads `rank`, rank + cluster, ..
    constexpr int W = HD / 32;
    const int last = (1 << log_cluster) - 1;
    for (int k = rank + (warp << log_cluster); k < nh; k += kWinWarps << log_cluster) {
        float m[8], l[8], v[8][W], top = -INFINITY, sum = 0.f, acc[W] = {0.f};
#pragma unroll
        for (int r = 0; r < 8; ++r) {                    // every load in flight at once
            load_from(mine_ml + 2 * k, min(r, last), m[r], l[r]);
            load_from(mine + k * HD + W * lane, min(r, last), v[r]);
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) top = fmaxf(top, m[r]);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (r > last || (m[r] == -INFINITY && l[r] == 0.f)) continue;     // no tiles there
            const float f = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - top);
            sum = fmaf(l[r], f, sum);
#pragma unroll
            for (int i = 0; i < W; ++i) acc[i] = fmaf(v[r][i], f, acc[i]);
        }
        const float inv = sum != 0.f ? p.out_scale / sum : 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) store_from_float<QT>(p.out, (row0 + k) * HD + W * lane + i, acc[i] * inv);
    }
    __syncwarp();
    cluster_sync();                                      // what the others read stays until they have
}

// CTAs of a cluster (and stages of the ring), by what a launch costs in rounds of tiles: rounds of
// resident CTAs, each of a CTA's tiles and kWinStart for its start and its end (and as much again for a
// cluster's meeting).  Measured (us): one sequence under 1,024 tokens 5.1 in clusters of eight; 80 units of
// 4,096 27.6 in pairs, 35.5 in fours; 160 units of 4,096 49.6 alone, 60.2 in pairs; FP8, 512 units of 4,096
// 94 in fours of four stages (three CTAs an SM), 85 alone of three (four an SM), 320 units of 1,024 15.0
// and 18.6 alone of four and of three.
constexpr int kWinStart = 3;

template <typename QT, typename KT, int HD>
cudaError_t launch_decode_window(const DecodeParams& p, cudaStream_t stream) {
    using C = WinCfg<QT, KT, HD>;
    static int resident[2][64] = {{0}};                  // with all stages, with the fewest
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    auto kernel = decode_window_kernel<QT, KT, HD>;
    if (resident[1][dev] == 0) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(C::NSTAGE));
        if (err != cudaSuccess) return err;
        int sms = 0;
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (err != cudaSuccess) return err;
        for (int i = 0; i < 2; ++i) {
            int per_sm = 0;
            err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kWinThreads,
                                                                C::smem(i ? C::FEWEST : C::NSTAGE));
            if (err != cudaSuccess) return err;
            resident[i][dev] = (per_sm > 0 ? per_sm : 1) * sms;
        }
    }
    CUtensorMap tk{}, tv{};
    const long long rows = (long long)p.num_blocks * p.num_kv_heads * p.block_size;
    if (!C::FP4 && (!encode_pool_map(&tk, p.k_cache, HD, C::ELEM_BYTES, rows, p.block_size) ||
                    !encode_pool_map(&tv, p.v_cache, HD, C::ELEM_BYTES, rows, p.block_size)))
        return cudaErrorInvalidValue;
    const int64_t units = (int64_t)p.num_seqs * p.num_kv_heads * p.nsub;
    const int64_t tiles = ((int64_t)p.max_seen + kWinTile - 1) / kWinTile;
    int log_cluster = 0, stages = C::NSTAGE;
    int64_t least = INT64_MAX;
    for (int i = 0; i <= (C::FEWEST < C::NSTAGE); ++i)
        for (int k = 0; k <= 3 && (k == 0 || tiles >= 1 << k); ++k) {
            const int64_t rounds = ((units << k) + resident[i][dev] - 1) / resident[i][dev];
            const int64_t cost = rounds * (((tiles + (1 << k) - 1) >> k) + kWinStart * (k ? 2 : 1));
            if (cost < least) {
                least = cost;
                log_cluster = k;
                stages = i ? C::FEWEST : C::NSTAGE;
            }
        }
    if ((units << log_cluster) > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = 1 << log_cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units << log_cluster), 1, 1);
    cfg.blockDim = dim3(kWinThreads, 1, 1);
    cfg.dynamicSmemBytes = C::smem(stages);
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, log_cluster, stages, 0x10010u, 0x1001u, tk, tv);   // 2^4 + 2^16, 1 + 2^12
}

}  // namespace
}  // namespace pkv
