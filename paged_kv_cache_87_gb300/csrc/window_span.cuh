// window_span.cuh -- what a token under a sliding window sees of its context.
//
// The token at position n - 1 of a context of n tokens sees the last `window` of them, from
// low = max(0, n - window) on, and the first `sinks`.  Blocks that hold nothing of either are left
// out, so a kernel walks a shorter, virtual context: the blocks of the sinks, then the window's.
// Of its tokens those between the last sink and the window's first token are hidden: what is left
// of the sinks' last block and the beginning of the window's first, less than a block each, so every
// block of the virtual context holds a token that is seen.
#pragma once

#include <stdint.h>

namespace pkv {

struct WindowSpan {
    int tokens;               // of the virtual context
    int sink_blocks;          // its blocks before the window's
    int skip_blocks;          // blocks of the context that are left out behind them
    int hide_lo, hide_hi;     // its tokens that are hidden: [hide_lo, hide_hi)
};

__host__ __device__ __forceinline__ WindowSpan window_span(int n, int window, int sinks, int log_block) {
    WindowSpan w{n, 0, 0, 0, 0};
    const int low = n - window;                       // window >= 1: below n
    if (low <= 0) return w;
    const int kept = sinks < low ? sinks : low;       // the sinks that the window leaves out
    const int first = low >> log_block;               // the window's first block
    w.sink_blocks = kept <= 0 ? 0 : ((kept - 1) >> log_block) + 1;
    w.skip_blocks = first > w.sink_blocks ? first - w.sink_blocks : 0;
    w.tokens = n - (w.skip_blocks << log_block);
    w.hide_lo = kept;
    w.hide_hi = low - (w.skip_blocks << log_block);
    return w;
}

// The entry of a sequence's block table that holds block j of the virtual context.
__device__ __forceinline__ int window_entry(const WindowSpan& w, int j) {
    return j < w.sink_blocks ? j : j + w.skip_blocks;
}

// Tokens of the longest virtual context, at most.
inline int window_most(int max_context_len, int window, int sinks, int block) {
    const int64_t most = (int64_t)window + block - 1 + ((int64_t)sinks + block - 1) / block * block;
    return most < max_context_len ? (int)most : max_context_len;
}

}  // namespace pkv
