"""Pins of the plain windowed attention: torch's masked attention, closed forms, the plain decode."""
import numpy as np
import pytest
import torch

from oracle import fp4, window


@pytest.mark.parametrize("n,m,w,sinks", [(1, 1, 1, 0), (9, 1, 4, 2), (17, 17, 5, 3), (40, 7, 100, 0),
                                         (33, 12, None, 0), (30, 30, 1, 1), (25, 6, 3, 40)])
def test_attention_is_torchs_under_a_mask(n, m, w, sinks):
    rng = np.random.default_rng(n * 100 + m)
    q, k, v = (rng.standard_normal(s) for s in ((m, 6, 8), (2, n, 8), (2, n, 8)))
    mask = torch.zeros(m, n, dtype=torch.bool)
    for i in range(m):
        p = n - m + i
        for t in range(p + 1):
            mask[i, t] = w is None or p - t < w or t < sinks
    t = lambda a: torch.from_numpy(a)
    ref = torch.nn.functional.scaled_dot_product_attention(
        t(q).transpose(0, 1), t(k).repeat_interleave(3, 0), t(v).repeat_interleave(3, 0),
        attn_mask=mask, scale=0.3).transpose(0, 1)
    assert np.abs(window.attention(q, k, v, 0.3, w, sinks) - ref.numpy()).max() < 1e-12


def test_a_window_of_one_sees_itself_and_a_wide_one_everything():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal(s) for s in ((5, 4, 8), (2, 20, 8), (2, 20, 8)))
    one = window.attention(q, k, v, 0.3, 1, 0)
    assert np.allclose(one, np.repeat(v[:, 15:].transpose(1, 0, 2), 2, 1))
    assert np.allclose(window.attention(q, k, v, 0.3, 20, 0), window.attention(q, k, v, 0.3))
    assert np.allclose(window.attention(q[4:], k, v, 0.3)[0], fp4.attention(q[4], k, v, 0.3))
    assert (window.attention(q[:1], k[:, :0], v[:, :0], 0.3, 3, 1) == 0).all()


def test_rows_that_nothing_sees_may_hold_anything():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal(s) for s in ((3, 2, 8), (1, 30, 8), (1, 30, 8)))
    want = window.attention(q, k, v, 0.3, 4, 2)
    k[:, 2:24], v[:, 2:24] = np.nan, np.inf              # 30 - 3 - 4 + 1 = 24 is the first in the window
    assert (window.attention(q, k, v, 0.3, 4, 2) == want).all()


def _virtual(n, w, sinks, B):
    """The virtual context by its definition: blocks that hold a token that is seen, in order."""
    seen = window.seen(n, 1, w, sinks)[0]
    blocks = sorted({t // B for t in np.flatnonzero(seen)} | ({(n - 1) // B}))
    tokens = [t for b in blocks for t in range(b * B, min(n, b * B + B))]
    return blocks, tokens, seen[tokens]


@pytest.mark.parametrize("B", [8, 16, 32])
def test_virtual_contexts(B, tmp_path):
    """window_span() of the kernels, compiled for the host, against the definition."""
    import ctypes
    import os
    import subprocess
    import paged_kv_cache_87_gb300 as pkg
    src = os.path.join(os.path.dirname(pkg.__file__), "csrc", "window_span.cuh")
    c = tmp_path / "span.cpp"
    c.write_text('#define __host__\n#define __device__\n#define __forceinline__ inline\n'
                 f'#include "{src}"\nextern "C" void span(int n, int w, int s, int b, int* o) {{\n'
                 'pkv::WindowSpan x = pkv::window_span(n, w, s, b);\n'
                 'o[0] = x.tokens; o[1] = x.sink_blocks; o[2] = x.skip_blocks; o[3] = x.hide_lo; o[4] = x.hide_hi; }\n'
                 'extern "C" int entry(int n, int w, int s, int b, int j) {\n'
                 'return pkv::window_entry(pkv::window_span(n, w, s, b), j); }\n'
                 'extern "C" int most(int n, int w, int s, int b) { return pkv::window_most(n, w, s, b); }\n')
    so = str(tmp_path / "span.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-o", so, str(c)], check=True)
    lib = ctypes.CDLL(so)
    log = {8: 3, 16: 4, 32: 5}[B]
    rng = np.random.default_rng(B)
    cases = [(int(rng.integers(1, 400)), int(rng.integers(1, 300)), int(rng.integers(0, 80))) for _ in range(400)]
    cases += [(n, w, s) for n in (1, B, B + 1, 5 * B) for w in (1, B, 2 * B, 10 ** 6) for s in (0, 1, B, 10 ** 6)]
    for n, w, s in cases:
        o = (ctypes.c_int * 5)()
        lib.span(n, w, s, log, o)
        blocks, tokens, seen = _virtual(n, w, s, B)
        got = [t for t in range(o[0])]
        assert [lib.entry(n, w, s, log, j) for j in range(-(-o[0] // B))] == blocks, (n, w, s)
        assert len(got) == len(tokens)
        assert [not o[3] <= t < o[4] for t in got] == seen.tolist(), (n, w, s)
        assert o[0] <= lib.most(max(n, 400), w, s, B)
    big = 2 ** 31 - 1
    o = (ctypes.c_int * 5)()
    lib.span(100, big, big, log, o)
    assert list(o) == [100, 0, 0, 0, 0] and lib.most(big, big, big, B) == big


def test_chunk_spans(tmp_path):
    """chunk_span() of the planner, compiled for the host: its blocks are those that hold a token that
    a row sees, in order, and what it hides of them is what no row sees."""
    import ctypes
    import os
    import re
    import subprocess
    import paged_kv_cache_87_gb300 as pkg
    text = open(os.path.join(os.path.dirname(pkg.__file__), "csrc", "chunk_attention.cuh")).read()
    body = re.search(r"struct ChunkSpan \{.*?\n\};", text, re.S).group(0) + "\n" + \
        re.search(r"__host__ __device__ __forceinline__ ChunkSpan chunk_span.*?\n\}\n", text, re.S).group(0)
    c = tmp_path / "span.cpp"
    c.write_text('#define __host__\n#define __device__\n#define __forceinline__ inline\n'
                 'constexpr int kChunkTile = 128;\n' + body +
                 'extern "C" void span(int p, int e, int w, int s, int b, int* o) {\n'
                 'ChunkSpan x = chunk_span(p, e, w, s, b);\n'
                 'o[0] = x.skip; o[1] = x.sink_blocks; o[2] = x.low; o[3] = x.kv_end; o[4] = x.steps; }\n')
    so = str(tmp_path / "span.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-o", so, str(c)], check=True)
    lib = ctypes.CDLL(so)
    rng = np.random.default_rng(0)
    for _ in range(900):
        log = int(rng.integers(3, 6))
        B = 1 << log
        n = int(rng.integers(1, 2000))
        m = int(rng.integers(1, min(n, 300) + 1))
        w, s = int(rng.integers(1, 700)), int(rng.integers(0, 400))
        o = (ctypes.c_int * 5)()
        lib.span(n - m, n, w, s, log, o)
        skip, sink_blocks, low, kv_end, steps = o
        assert skip % B == 0 and steps == -(-kv_end // 128)
        seen = window.seen(n, m, w, s)
        blocks = [j if j < sink_blocks else j + skip // B for j in range(-(-kv_end // B))]
        assert blocks == sorted(set((np.flatnonzero(seen.any(0)) // B).tolist())), (n, m, w, s)
        # every row, in the virtual context: the mask that the kernel forms from its position there
        v = np.arange(kv_end)
        t = np.array([blocks[x // B] * B + x % B for x in v])
        pos = np.arange(n - m, n)[:, None] - skip
        mine = (v <= pos) & ((v > pos - w) | (v < s))
        assert (mine == seen[:, t]).all()
        assert (((v < s) | (v >= low)) == seen[:, t].any(0)).all()
