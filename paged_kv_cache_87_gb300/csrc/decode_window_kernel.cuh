// decode_window_kernel.cuh -- decode under a sliding window for 16-bit queries, in one launch:
// o = sum_t softmax_t(scale q.k_t) v_t over the tokens of the virtual context of window_span.cuh (the
// sinks' blocks, then the window's).
//
// A window bounds every unit (sequence, kv head, eight query heads), so there is nothing to plan: a
// cluster of 1, 2, 4, 8 or 16 CTAs takes a unit, an equal run of its 64-token tiles each, and joins its
// states through distributed shared memory.  A CTA is a producer warp, which fills a ring of tiles
// (TMA boxes through the block table, under the swizzle of a row's slices: 128 bytes, FP8 of 64 dims 64; 4 bits:
// bulk copies, unswizzled, as decode_fp4_kernel.cuh takes them), and four consumer warps, 16 tokens of every tile each (five warps
// spread over all four sub-partitions).  The products are row_tiles.cuh's.  Tokens that are hidden or past
// the context are masked in S and their rows of V zeroed in shared memory, by the warp that multiplies them.
//
// Measured (us; of the bytes' time at 6,792 GB/s): 256 sequences of 64 - 32k, 32 / 8 heads, d 128, bf16 under
// 1,024 + 4: 115 (1.0); 64 of 4k - 131k, 64 / 8, FP8 under 4,096 + 16: 85 (0.94), of 64 dims under 4,096: 45 (0.89),
// all bound by HBM; over 4 bits 256 under 1,024: 71 (0.64), nothing full (2.65 of 4 instructions a clock, DRAM 53 %):
// chains of dependent widening, products and softmax in four warps a CTA; one sequence under 1,024: 5.3 (0.11), bound by the latency of length, table, first tile and the
// cluster's meeting.
#pragma once

#include <atomic>
#include <mutex>

#include "row_tiles.cuh"
#include "window_span.cuh"

namespace pkv {
namespace {

template <typename QT, typename KT, int HD>
__global__ void __launch_bounds__(kRowThreads, (TileCfg<QT, KT, HD, 1>::CTAS)) decode_window_kernel(
    DecodeParams p, int log_cluster, int stages, uint32_t even, uint32_t odd, const __grid_constant__ CUtensorMap tmK,
    const __grid_constant__ CUtensorMap tmV) {
    using C = TileCfg<QT, KT, HD, 1>;
    extern __shared__ uint8_t smem_raw[];
    // every CTA of a cluster places its state alike: the offset to the boundary is the same
    uint8_t* smem = smem_raw + (-smem_addr(smem_raw) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + C::NSTAGE;
    uint8_t* ring = smem + C::OFF_RING;
    float* mine = reinterpret_cast<float*>(smem + C::OFF_MINE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kRowWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int logB = p.log_block, upi = p.num_kv_heads * p.nsub;
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
            for (int i = threadIdx.x; i < nh * HD; i += kRowThreads) store_from_float<QT>(p.out, row0 * HD + i, 0.f);
        return;
    }
    const WindowSpan span = window_span(n, p.window, p.sinks, logB);
    const int tiles = (span.tokens - 1) / kRowTile + 1;
    const int a = (int)((int64_t)tiles * rank >> log_cluster), end = (int)((int64_t)tiles * (rank + 1) >> log_cluster);

    if (warp == kRowWarps) {
        // ======================= producer warp =======================
        tile_producer<C, HD>(p.k_cache, p.v_cache, &tmK, &tmV, p.block_tables + (int64_t)s * p.max_blocks,
                             [&](int j) { return window_entry(span, j); }, span.tokens, a, end, logB, p.num_kv_heads,
                             kvh, p.num_blocks, stages, full, empty, ring, p.status);
        if (log_cluster) {
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
        return;
    }

    // ========================= consumer warps =========================
    const TileLane<C, HD> w(p.block_size, logB);
    uint32_t qf[1][C::KSTEPS][2];                // Q^T fragments of head g
    float qs0 = p.qk_scale_log2, qs1 = qs0;      // logit scales of heads 2c and 2c + 1
    tile_query<C, QT>(w, static_cast<const uint16_t*>(p.q) + (row0 + w.g) * HD, w.g < nh, qf[0], qs0, qs1);
    float o[1][C::MTILES][4];
#pragma unroll
    for (int mt = 0; mt < C::MTILES; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][mt][e] = 0.f;
    float m[1][2] = {{-INFINITY, -INFINITY}}, l[1][2] = {{0.f, 0.f}};    // of heads 2c and 2c + 1
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = a; t < end; ++t) {
        if (!mbar_wait(&full[stage], phase)) {
            set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
            ok = false;
            break;
        }
        uint8_t* sb = ring + stage * C::STAGE_BYTES;
        // this warp's rows: valid ones, hidden ones
        const int t0 = t * kRowTile + 16 * warp;
        const int nv = span.tokens - t0, ha = span.hide_lo - t0, hb = span.hide_hi - t0;
        if (nv > 0) {
            auto seen = [&](int r) { return r < nv && (r < ha || r >= hb); };
            const bool part = nv < 16 || (ha < hb && ha < 16 && hb > 0);
            if (!C::FP4 && part) tile_zero_rows(w, sb, seen);
            float x[1][4] = {{0.f, 0.f, 0.f, 0.f}};
            tile_scores(w, sb, [&](int, int k) { return make_uint2(qf[0][k][0], qf[0][k][1]); }, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[0][e] *= e & 1 ? qs1 : qs0;
            if (part) {
                if (!seen(w.g)) x[0][0] = x[0][1] = -INFINITY;
                if (!seen(w.g + 8)) x[0][2] = x[0][3] = -INFINITY;
            }
            uint32_t b[1][2];
            tile_softmax<C>(x, m, l, o, b);
            tile_weigh(w, sb, part, seen, even, odd, b, o);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
    }
    tile_finish<C, QT>(w, ring, mine, rank, 1 << log_cluster, a < end && ok, nh, p.out_scale, p.out,
                       [&](int k) { return (row0 + k) * HD; }, m, l, o);
    if (!ok) mbar_let_land(full, stages);
}

// CTAs of a cluster (and stages of the ring), by what a launch costs in rounds of tiles: rounds of
// resident CTAs, each of a CTA's tiles and kWinStart for its start and its end (and as much again for a
// cluster's meeting).  Measured (us): one sequence under 1,024 tokens 5.1 in clusters of eight; 80 units of
// 4,096 27.6 in pairs, 35.5 in fours; 160 units of 4,096 49.6 alone, 60.2 in pairs; 320 of 1,024 33.8 in three
// stages, 27.4 in two; FP8, 512 units of 4,096 94 in fours of four stages (three CTAs an SM), 85 alone of three
// (four an SM), 320 units of 1,024 15.0 and 18.6 alone of four and of three.
constexpr int kWinStart = 3;
// Sixteen CTAs a cluster are more than every device has to offer (and are asked for): units of 64 tiles or more take
// them where all units' clusters are resident at once, which is fewer than their CTAs would be, since a cluster
// lies within a GPC.  One sequence, 8 / 1 heads, bf16, in eights and sixteens: 1,024 tokens 4.8 and 4.9 us, 2,048 6.3
// and 5.7 (16 units, FP8, 7.5 and 8.8), 4,096 9.0 and 7.1 (10.3 and 10.3), 131,072 177 and 92 (64 / 8 heads 185 and
// 97; the plain decode of as many 138); where they take a second round, 16 units of 131,072, 185 and 188.
constexpr int kWinWide = 64;

// What a device holds at once, with all stages of the ring and with the fewest: CTAs, clusters of sixteen.
struct WindowRoom {
    int ctas[2], wide[2];
};

// Asked for once a device; several threads may be the first.
template <typename QT, typename KT, int HD>
cudaError_t window_room(int dev, WindowRoom* out) {
    using C = TileCfg<QT, KT, HD, 1>;
    static std::mutex lock;
    static std::atomic<bool> known[64];
    static WindowRoom rooms[64];
    if (!known[dev].load(std::memory_order_acquire)) {
        const std::lock_guard<std::mutex> held(lock);
        auto kernel = decode_window_kernel<QT, KT, HD>;
        cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(C::NSTAGE));
        if (err != cudaSuccess) return err;
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);     // sixteen
        if (err != cudaSuccess) return err;
        int sms = 0;
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (err != cudaSuccess) return err;
        for (int i = 0; i < 2; ++i) {
            int per_sm = 0;
            err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kRowThreads,
                                                                C::smem(i ? C::FEWEST : C::NSTAGE));
            if (err != cudaSuccess) return err;
            cudaLaunchAttribute of16[1];
            of16[0].id = cudaLaunchAttributeClusterDimension;
            of16[0].val.clusterDim.x = 16;
            of16[0].val.clusterDim.y = of16[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t at = {};
            at.gridDim = dim3(16, 1, 1);
            at.blockDim = dim3(kRowThreads, 1, 1);
            at.dynamicSmemBytes = C::smem(i ? C::FEWEST : C::NSTAGE);
            at.attrs = of16;
            at.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&rooms[dev].wide[i], kernel, &at) != cudaSuccess) {
                rooms[dev].wide[i] = 0;                  // (a device without them)
                (void)cudaGetLastError();
            }
            rooms[dev].ctas[i] = (per_sm > 0 ? per_sm : 1) * sms;
        }
        known[dev].store(true, std::memory_order_release);
    }
    *out = rooms[dev];
    return cudaSuccess;
}

template <typename QT, typename KT, int HD>
cudaError_t launch_decode_window(const DecodeParams& p, cudaStream_t stream) {
    using C = TileCfg<QT, KT, HD, 1>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    WindowRoom room;
    err = window_room<QT, KT, HD>(dev, &room);
    if (err != cudaSuccess) return err;
    auto kernel = decode_window_kernel<QT, KT, HD>;
    CUtensorMap tk{}, tv{};
    const long long rows = (long long)p.num_blocks * p.num_kv_heads * p.block_size;
    if (!C::FP4 && (!encode_pool_map(&tk, p.k_cache, HD, C::ELEM_BYTES, rows, p.block_size) ||
                    !encode_pool_map(&tv, p.v_cache, HD, C::ELEM_BYTES, rows, p.block_size)))
        return cudaErrorInvalidValue;
    const int64_t units = (int64_t)p.num_seqs * p.num_kv_heads * p.nsub;
    const int64_t tiles = ((int64_t)p.max_seen + kRowTile - 1) / kRowTile;
    int log_cluster = 0, stages = C::NSTAGE;
    int64_t least = INT64_MAX;
    for (int i = 0; i <= (C::FEWEST < C::NSTAGE); ++i)
        for (int k = 0; k <= 4 && (k == 0 || tiles >= 1 << k); ++k) {
            if (k == 4 && (tiles < kWinWide || units > room.wide[i])) break;
            const int64_t rounds = ((units << k) + room.ctas[i] - 1) / room.ctas[i];
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
    cfg.blockDim = dim3(kRowThreads, 1, 1);
    cfg.dynamicSmemBytes = C::smem(stages);
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, log_cluster, stages, 0x10010u, 0x1001u, tk, tv);   // 2^4 + 2^16, 1 + 2^12
}

}  // namespace
}  // namespace pkv
