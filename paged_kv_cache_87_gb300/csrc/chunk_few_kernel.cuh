// chunk_few_kernel.cuh -- the chunk attention of many sequences with few rows (a batch's chains of drafts,
// single tokens beside them): up to kChunkFewRows (new token, query head of the group) rows of a kv head.
//
// o(p) = sum_t softmax_t(scale q.k_t) v_t over what the token at p sees, as in chunk_kernel.cuh.  There a
// tcgen05 tile has 128 rows, of which such a sequence fills a sixth, and FP8 and 4 bits are widened through
// shared memory, whose bandwidth bounds it.  Here rows are the narrow side of mma.sync, as in the decodes:
// three sets of eight, widened in registers once for all sets (row_tiles.cuh).  A CTA takes a (sequence, kv
// head): one launch, nothing planned, no workspace.  Sequences with more rows leave at once; the chunk kernel,
// launched behind, takes those and leaves these.
//
// Contexts are not cut, so there have to be enough of them for the longest to end among the others (chunk_few in
// api.cu, with what was measured on either side), and single long ones are left to the chunk kernel (few_most).  Large ones (us, the chunk kernel alone | with this one), 5 tokens
// over 1,000 - 8,000, 32 / 8 heads, bf16 queries: FP8, d 128, 200 sequences 541 | 380, 100 275 | 228; 4 bits, d 128,
// 588 | 355, 290 | 210; d 64, 200 sequences: FP8 453 | 208, 4 bits 453 | 226, 16 bits 412 | 254.  3 tokens under a window of 1,024 + 4, 256 sequences:
// FP8 219 | 154, 16 bits of 64 dims 194 | 102.  16 bits of 128 dims, where the chunk kernel widens nothing,
// 468 | 462, 236 | 262: not taken.
// What bounds it: 450 instructions and 48 products a warp and 16 tokens, with two CTAs' warps an SM (three of 64
// dims) to hide their latencies (FP8: 0.36 of an instruction a clock and sub-partition, tensor pipe 35 %, HBM
// 56 %); three sets' sums of O leave no registers for more.  Q^T comes from shared memory for the same reason:
// in registers it spilled (32 sequences of 5 over 4,096, FP8: 186 us, 82 from shared memory, 69 with one vote
// of the warp for all sets' maxima).
// Tried and not kept: clusters that cut every context alike (drafts of 32 sequences 107 - 144 us, the chunk kernel
// 92), or as its length asks, the rest of the cluster leaving (112; 155 against 69 where nothing is cut).
#pragma once

#include <atomic>

#include "chunk_attention.cuh"
#include "row_tiles.cuh"

namespace pkv {
namespace {

constexpr int kFewSets = kChunkFewRows / 8;
template <typename QT, typename KT, int HD>
__global__ void __launch_bounds__(kRowThreads, (TileCfg<QT, KT, HD, kFewSets>::CTAS)) chunk_few_kernel(
    ChunkParams p, uint32_t even, uint32_t odd, const __grid_constant__ CUtensorMap tmK,
    const __grid_constant__ CUtensorMap tmV) {
    constexpr int N = kFewSets;
    using C = TileCfg<QT, KT, HD, N>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_addr(smem_raw) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + C::NSTAGE;
    uint8_t* ring = smem + C::OFF_RING;
    uint2* qs_frag = reinterpret_cast<uint2*>(smem + C::OFF_Q);              // Q^T's fragments, [set][k-step][lane]
    int64_t* place = reinterpret_cast<int64_t*>(smem + C::OFF_ROWS);       // a row's place in q and out
    int* at = reinterpret_cast<int*>(place + 8 * N);                       // its token in the virtual context
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, logB = p.log_block;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NSTAGE; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kRowWarps);
        }
        fence_mbar_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    const int s = blockIdx.x / p.num_kv_heads, kvh = blockIdx.x - s * p.num_kv_heads;
    const int q0 = p.query_start[s], q1 = p.query_start[s + 1], ctx = p.context_lens[s];
    const int64_t n64 = (int64_t)q1 - q0, cap = min((int64_t)p.max_context_len, (int64_t)p.max_blocks * p.block_size);
    const bool good = n64 >= 0 && q0 >= 0 && q1 <= p.total_q && ctx >= n64 && ctx <= cap;
    if (kvh == 0 && threadIdx.x == 0 &&
        (!good || (s == 0 && q0 != 0) || (s == p.num_seqs - 1 && q1 != p.total_q)))
        set_status(p.status, PKV_DEV_BAD_CONTEXT);
    if (!good || n64 == 0 || n64 * p.group > kChunkFewRows) return;
    const int n = (int)n64;
    const int rows = n * p.group, first = ctx - n;
    const ChunkSpan span = chunk_span(first, ctx, p.window, p.sinks, logB);
    if (p.few_ctas && span.kv_end > kChunkFewAlone) {          // too long for this kernel?
        int most;
        if (p.self_plan) {                                     // up to 32 sequences, one a lane
            int walked = 0;
            if (lane < p.num_seqs) {
                const int a = p.query_start[lane], c = p.context_lens[lane];
                const int64_t r = (int64_t)p.query_start[lane + 1] - a;
                if (r >= 0 && a >= 0 && a + r <= p.total_q && c >= r && c <= cap) walked = few_tokens(p, r, c);
            }
            most = few_most(p, few_sum(walked));
        } else {
            most = p.head->few_most;
        }
        if (span.kv_end > most) return;
    }
    if (threadIdx.x < 8 * N) {
        const int r = min((int)threadIdx.x, rows - 1), token = r / p.group;
        place[threadIdx.x] = (((int64_t)q0 + token) * p.num_q_heads + kvh * p.group + (r - token * p.group)) * HD;
        at[threadIdx.x] = first + token - span.skip;
    }
    __syncthreads();
    const int tiles = (span.kv_end - 1) / kRowTile + 1;

    if (warp == kRowWarps) {
        tile_producer<C, HD>(p.k_cache, p.v_cache, &tmK, &tmV, p.block_tables + (int64_t)s * p.max_blocks,
                             [&](int j) { return j < span.sink_blocks ? j : j + (span.skip >> logB); }, span.kv_end, 0,
                             tiles, logB, p.num_kv_heads, kvh, p.num_blocks, C::NSTAGE, full, empty, ring, p.status);
        return;
    }

    const TileLane<C, HD> w(p.block_size, logB);
    float qs[N][2], m[N][2], l[N][2], o[N][C::MTILES][4];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        qs[i][0] = qs[i][1] = p.qk_scale_log2;
        m[i][0] = m[i][1] = -INFINITY;
        l[i][0] = l[i][1] = 0.f;
        uint32_t qf[C::KSTEPS][2];
        tile_query<C, QT>(w, static_cast<const uint16_t*>(p.q) + place[8 * i + w.g], 8 * i + w.g < rows, qf, qs[i][0],
                          qs[i][1]);
        if (warp == i)
#pragma unroll
            for (int k = 0; k < C::KSTEPS; ++k) qs_frag[(i * C::KSTEPS + k) * 32 + lane] = make_uint2(qf[k][0], qf[k][1]);
#pragma unroll
        for (int mt = 0; mt < C::MTILES; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][mt][e] = 0.f;
    }
    static_assert(N <= kRowWarps, "a warp a set");
    named_bar_sync(1, kRowWarps * 32);
    const int first_at = at[0], last_at = span.kv_end - 1;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = 0; t < tiles; ++t) {
        if (!mbar_wait(&full[stage], phase)) {
            set_status(p.status, PKV_DEV_WAIT_TIMEOUT);
            ok = false;
            break;
        }
        uint8_t* sb = ring + stage * C::STAGE_BYTES;
        const int t0 = t * kRowTile + 16 * warp;                           // this warp's first token
        if (t0 <= last_at) {
            // tokens that any row sees; and whether there are some that not every row sees
            auto seen = [&](int r) { return t0 + r <= last_at && (t0 + r >= span.low || t0 + r < p.sinks); };
            const bool part = t0 + 15 > first_at || (t0 <= last_at - p.window && t0 + 15 >= p.sinks);
            if (!C::FP4 && part) tile_zero_rows(w, sb, seen);
            float x[N][4];
#pragma unroll
            for (int i = 0; i < N; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
            tile_scores(w, sb, [&](int i, int k) { return qs_frag[(i * C::KSTEPS + k) * 32 + lane]; }, x);
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][e] *= qs[i][e & 1];
            if (part) {
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int tok = t0 + w.g + 8 * (e >> 1), pos = at[8 * i + 2 * w.c + (e & 1)];
                        if (tok > pos || (tok <= pos - p.window && tok >= p.sinks)) x[i][e] = -INFINITY;
                    }
            }
            uint32_t b[N][2];
            tile_softmax<C>(x, m, l, o, b);
            tile_weigh(w, sb, part, seen, even, odd, b, o);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == C::NSTAGE) { stage = 0; phase ^= 1u; }
    }
    tile_finish<C, QT>(w, ring, nullptr, 0, 1, ok, rows, p.out_scale, p.out,
                       [&](int k) { return place[k]; }, m, l, o);
    if (!ok) mbar_let_land(full, C::NSTAGE);
}

template <typename QT, typename KT, int HD>
cudaError_t launch_chunk_few(const ChunkParams& p, cudaStream_t stream) {
    using C = TileCfg<QT, KT, HD, kFewSets>;
    static std::atomic<bool> attr_set[64];            // (several threads may be the first)
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    auto kernel = chunk_few_kernel<QT, KT, HD>;
    if (!attr_set[dev]) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(C::NSTAGE));
        if (err != cudaSuccess) return err;
        attr_set[dev] = true;
    }
    CUtensorMap tk{}, tv{};
    const long long rows = (long long)p.num_blocks * p.num_kv_heads * p.block_size;
    if (!C::FP4 && (!encode_pool_map(&tk, p.k_cache, HD, C::ELEM_BYTES, rows, p.block_size) ||
                    !encode_pool_map(&tv, p.v_cache, HD, C::ELEM_BYTES, rows, p.block_size)))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attrs[1];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.num_seqs * p.num_kv_heads), 1, 1);
    cfg.blockDim = dim3(kRowThreads, 1, 1);
    cfg.dynamicSmemBytes = C::smem(C::NSTAGE);
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, 0x10010u, 0x1001u, tk, tv);      // 2^4 + 2^16, 1 + 2^12
}

template <typename QT>
cudaError_t launch_chunk_few_q(const ChunkParams& p, int head_dim, pkv_dtype kv, cudaStream_t s) {
    if (kv == PKV_FP8_E4M3)
        return head_dim == 128 ? launch_chunk_few<QT, E4M3, 128>(p, s) : launch_chunk_few<QT, E4M3, 64>(p, s);
    if (kv == PKV_FP4_E2M1)
        return head_dim == 128 ? launch_chunk_few<QT, E2M1, 128>(p, s) : launch_chunk_few<QT, E2M1, 64>(p, s);
    return launch_chunk_few<QT, QT, 64>(p, s);
}

}  // namespace
}  // namespace pkv
