"""Python binding of libpagedkv.so (C ABI: include/pagedkv.h).

Argument marshalling only: shapes, dtypes and the stream are read off torch
tensors and passed as plain pointers and sizes -- for the calls of a serving
step in the extension module _marshal (csrc/host/marshal.cc, compiled for the torch that is
installed), for the rest through ctypes; every step of the hot path runs in the library's CUDA
kernels.  There is no CPU fallback: if the library or the module cannot be loaded the calls raise.

Calls run on the current device, where their tensors have to be (the extension module refuses
others), and on its current stream or the one given.  What a call allocates for a stream other
than the current one is that stream's memory, held until the current stream is through too.

Functions carry the C names:
  pkv_decode_workspace_bytes, pkv_paged_decode_attention,
  pkv_paged_decode_attention_prefix, pkv_paged_decode_attention_noalloc,
  pkv_paged_decode_attention_window, pkv_paged_chunk_attention, pkv_reshape_and_cache, pkv_copy_blocks,
  pkv_gather_cache, pkv_qk_norm_rope, pkv_qk_norm_rope_and_cache,
  pkv_get_device_status, pkv_status_string, pkv_version,
and the host block manager pkv_bm_* (wrapped by ``BlockManager``).
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpagedkv.so")

PKV_F32, PKV_F16, PKV_BF16, PKV_FP8_E4M3, PKV_FP4_E2M1 = range(5)
(PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE, PKV_ERR_CUDA,
 PKV_ERR_OUT_OF_BLOCKS) = range(6)
(DEV_BAD_BLOCK_ID, DEV_BAD_CONTEXT, DEV_BAD_SLOT, DEV_BAD_PAIR, DEV_WAIT_TIMEOUT,
 DEV_BAD_POSITION) = (0x1, 0x2, 0x4, 0x8, 0x10, 0x20)

# ctypes signatures of every exported symbol
_P, _I, _L, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
_SIGNATURES = {
    "pkv_gather_cache": (ctypes.c_int, [_P] * 5 + [_I] * 8 + [_F, _I, _P, _P, _P]),
    "pkv_qk_norm_rope": (
        ctypes.c_int, [_P, _L, _P, _L, _P, _P, _I, _F, _P, _I, _I, _I, _P] + [_I] * 5 +
        [_P, _L, _P, _L, _P]),
    "pkv_qk_norm_rope_and_cache": (
        ctypes.c_int, [_P, _L, _P, _L, _P, _L, _P, _P, _I, _F, _P, _I, _I, _I, _P] + [_I] * 5 +
        [_P, _L, _P, _P, _P, _I, _I, _I, _F, _P]),
    "pkv_decode_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 6 + [ctypes.c_int]),
    "pkv_paged_decode_attention": (
        ctypes.c_int,
        [ctypes.c_void_p] * 5 + [ctypes.c_int] * 8 + [ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                                     ctypes.c_float, ctypes.c_void_p,
                                                     ctypes.c_size_t, ctypes.c_void_p,
                                                     ctypes.c_void_p]),
    "pkv_paged_decode_attention_prefix": (
        ctypes.c_int,
        [ctypes.c_void_p] * 5 + [ctypes.c_int] * 8 + [ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                                     ctypes.c_float, ctypes.c_void_p,
                                                     ctypes.c_size_t, ctypes.c_void_p,
                                                     ctypes.c_void_p]),
    "pkv_decode_window_workspace_bytes": (ctypes.c_size_t, [_I] * 10),
    "pkv_paged_decode_attention_window": (
        ctypes.c_int, [_P] * 5 + [_I] * 10 + [_F, _I, _I, _F, _P, ctypes.c_size_t, _P, _P]),
    "pkv_chunk_workspace_bytes": (ctypes.c_size_t, [_I] * 6),
    "pkv_paged_chunk_attention": (
        ctypes.c_int, [_P] * 6 + [_I] * 11 + [_F, _I, _I, _F, _P, ctypes.c_size_t, _P, _P]),
    "pkv_multi_query_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int]),
    "pkv_paged_multi_query_attention": (
        ctypes.c_int,
        [ctypes.c_void_p] * 6 + [ctypes.c_int] * 9 + [ctypes.c_float, ctypes.c_int,
                                                      ctypes.c_int, ctypes.c_float,
                                                      ctypes.c_void_p, ctypes.c_size_t,
                                                      ctypes.c_void_p, ctypes.c_void_p]),
    "pkv_paged_tree_attention": (
        ctypes.c_int,
        [ctypes.c_void_p] * 7 + [ctypes.c_int] * 9 + [ctypes.c_float, ctypes.c_int,
                                                      ctypes.c_int, ctypes.c_float,
                                                      ctypes.c_void_p, ctypes.c_size_t,
                                                      ctypes.c_void_p, ctypes.c_void_p]),
    "pkv_paged_decode_attention_noalloc": (
        ctypes.c_int,
        [ctypes.c_void_p] * 5 + [ctypes.c_int] * 8 + [ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                                     ctypes.c_float, ctypes.c_void_p,
                                                     ctypes.c_void_p]),
    "pkv_reshape_and_cache": (
        ctypes.c_int,
        [ctypes.c_void_p] * 5 + [ctypes.c_int] * 5 + [ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                                     ctypes.c_void_p]),
    "pkv_copy_blocks": (
        ctypes.c_int,
        [ctypes.c_void_p] * 3 + [ctypes.c_int] * 5 + [ctypes.c_int, ctypes.c_void_p]),
    "pkv_get_device_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint)]),
    "pkv_selftest_wait_bound": (ctypes.c_int, [ctypes.c_void_p]),
    "pkv_swap_blocks": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                       ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                       ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       ctypes.c_void_p]),
    "pkv_bm_create": (ctypes.c_void_p, [ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                        ctypes.c_int]),
    "pkv_bm_destroy": (None, [ctypes.c_void_p]),
    "pkv_bm_num_free": (ctypes.c_int, [ctypes.c_void_p]),
    "pkv_bm_refcount": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32]),
    "pkv_bm_add_sequence": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64]),
    "pkv_bm_fork": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64]),
    "pkv_bm_append_slot": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.POINTER(ctypes.c_int64),
                                          ctypes.POINTER(ctypes.c_int32),
                                          ctypes.POINTER(ctypes.c_int32)]),
    "pkv_bm_free_sequence": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64]),
    "pkv_bm_sequence": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                       ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                       ctypes.POINTER(ctypes.c_int64)]),
    "pkv_bm_prepare_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                           ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.POINTER(ctypes.c_int), ctypes.c_void_p,
                                           ctypes.c_int, ctypes.c_void_p]),
    "pkv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "pkv_version": (ctypes.c_int, []),
}

_lock = threading.Lock()
_lib = None
_calls = None   # the extension module


class PagedKVError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_text(status)} (status {status})")


def load(path: str = LIB_PATH):
    """Load the CUDA library (build it first with ``paged_kv_cache_87_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with "
                                   "`python -m paged_kv_cache_87_gb300.build` (needs nvcc)")
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                f = getattr(lib, name)
                f.restype, f.argtypes = res, args
            _lib = lib
        return _lib


def _marshal():
    """The extension module, loaded on first use (built with the library, for one torch)."""
    global _calls
    if _calls is None:
        load()
        path = os.path.join(_PKG, "_marshal.so")
        build = "build it with `python -m paged_kv_cache_87_gb300.build` (needs nvcc, g++ and Python's headers)"
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: {build}")
        try:
            from . import _marshal as module
        except ImportError as e:
            raise RuntimeError(f"{path} does not fit this torch ({torch.__version__}) or Python: {build}") from e
        if module.TORCH != torch.__version__:
            raise RuntimeError(f"{path} was built for torch {module.TORCH}, this is {torch.__version__}: {build}")
        module.set_error(PagedKVError)
        _calls = module
    return _calls


def status_text(status: int) -> str:
    return load().pkv_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != PKV_OK:
        raise PagedKVError(fn, status)


_TORCH_CODES = {torch.float32: PKV_F32, torch.float16: PKV_F16, torch.bfloat16: PKV_BF16,
                torch.float8_e4m3fn: PKV_FP8_E4M3, torch.uint8: PKV_FP8_E4M3}
_NAME_CODES = {"f32": PKV_F32, "f16": PKV_F16, "bf16": PKV_BF16, "e4m3": PKV_FP8_E4M3,
               "e2m1": PKV_FP4_E2M1}


def dtype_code(x) -> int:
    if isinstance(x, torch.Tensor):
        return _TORCH_CODES[x.dtype]
    if isinstance(x, torch.dtype):
        return _TORCH_CODES[x]
    if isinstance(x, str):
        return _NAME_CODES[x]
    return int(x)


def fp4_cache_shape(num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int) -> tuple:
    """Shape of a uint8 tensor that holds a 4-bit (PKV_FP4_E2M1) cache.  Its last two
    dims are one (block, kv head) tile, whose bytes include/pagedkv.h lays out."""
    return (num_blocks, num_kv_heads, block_size, head_dim // 2 + head_dim // 16)


_FP4_ROW_BYTES = {36: 64, 72: 128}   # bytes of a row of a 4-bit cache -> head_dim


def _cache_type(cache: torch.Tensor) -> tuple:
    """(element type code, head_dim) of a cache [NB, Hkv, B, row].  A uint8 cache is FP8
    unless its rows are 36 or 72 bytes: then it holds 4-bit codes and their scales."""
    row = cache.shape[3]
    if cache.dtype == torch.uint8 and row in _FP4_ROW_BYTES:
        return PKV_FP4_E2M1, _FP4_ROW_BYTES[row]
    return _TORCH_CODES[cache.dtype], row


def _one_type(k_cache: torch.Tensor, v_cache: torch.Tensor) -> None:
    if _TORCH_CODES.get(v_cache.dtype) != _TORCH_CODES[k_cache.dtype]:
        raise ValueError("k_cache and v_cache must have one element type")


def _stream_ptr(stream) -> int:
    if stream is None:   # the handle itself: building a Stream object costs 2.8 us a call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return int(stream.cuda_stream)


def _cuda(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t


def _fresh(like: torch.Tensor, stream, nbytes: int | None = None) -> torch.Tensor:
    """A new tensor like `like` (or of `nbytes` bytes) for a call on `stream`.  Where that is not
    the current stream, the memory comes from what torch's allocator keeps for `stream` -- a block
    that the current stream has dropped may still have its work in flight -- and is held until the
    current stream, where the caller reads it, is through as well."""
    shape, dtype = (like.shape, like.dtype) if nbytes is None else ((nbytes,), torch.uint8)
    if stream is None or int(stream.cuda_stream) == _stream_ptr(None):
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(_torch_stream(stream)):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _torch_stream(stream) -> torch.cuda.Stream:
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(stream.cuda_stream)
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


# ------------------------------------------------------------------ calls --

def pkv_decode_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                               block_size: int, max_context_len: int, kv_dtype) -> int:
    return int(load().pkv_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                 block_size, max_context_len,
                                                 dtype_code(kv_dtype)))


def pkv_paged_decode_attention(query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               block_tables: torch.Tensor, context_lens: torch.Tensor,
                               max_context_len: int, scale: float, kv_scale: float = 1.0,
                               workspace: torch.Tensor | None = None,
                               out: torch.Tensor | None = None, stream=None,
                               prefix: bool = False) -> torch.Tensor:
    """out[s, h] = softmax(scale * q[s, h] . K_s^T) V_s over context_lens[s] tokens.

    query [S, Hq, d]; k_cache / v_cache [NB, Hkv, B, d] (float8_e4m3fn or uint8
    for FP8; uint8 of fp4_cache_shape for 4 bits); block_tables int32 [S, max_blocks]; context_lens int32 [S].
    ``workspace`` (uint8, >= pkv_decode_workspace_bytes) is allocated if None.
    ``out`` has query's type, or is as many bytes in integers (larger ones are filled in part).
    ``prefix=True`` calls pkv_paged_decode_attention_prefix (shared prompts
    read once per group of sequences).
    """
    return (_calls or _marshal()).decode(query, k_cache, v_cache, block_tables, context_lens,
                                         max_context_len, scale, kv_scale, workspace, out,
                                         stream, prefix, False)


def pkv_decode_window_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                      head_dim: int, block_size: int, max_context_len: int,
                                      window: int, sinks: int, q_dtype, kv_dtype) -> int:
    """0 where the call needs none (most calls of 16-bit queries: include/pagedkv.h)."""
    return int(load().pkv_decode_window_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                        block_size, max_context_len, window, sinks,
                                                        dtype_code(q_dtype), dtype_code(kv_dtype)))


def pkv_paged_decode_attention_window(query: torch.Tensor, k_cache: torch.Tensor,
                                      v_cache: torch.Tensor, block_tables: torch.Tensor,
                                      context_lens: torch.Tensor, max_context_len: int,
                                      scale: float, window: int, sinks: int = 0,
                                      kv_scale: float = 1.0,
                                      workspace: torch.Tensor | None = None,
                                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pkv_paged_decode_attention of queries that see only the last ``window`` tokens of their
    context (their own among them) and its first ``sinks``.  Table entries of blocks that hold
    none of these are never read: such blocks may have been given back.  ``workspace`` is of
    pkv_decode_window_workspace_bytes; the other arguments are those of the plain call."""
    return (_calls or _marshal()).decode_window(query, k_cache, v_cache, block_tables, context_lens,
                                                max_context_len, scale, kv_scale, workspace, out,
                                                stream, False, False, window, sinks)


class PreparedCall:
    """One C-ABI call whose arguments (pointers, sizes, stream) were checked and
    marshalled once; calling it issues the same call again.

    For a serving loop that runs the same step on the same buffers every
    iteration: the per-call Python cost drops to one ctypes call.  The tensors
    behind the pointers are kept referenced here and must not be reallocated."""

    def __init__(self, name: str, args: tuple, keep: tuple = ()):
        self.name = name
        self._fn = getattr(load(), name)
        self._args = tuple(args)
        self._keep = keep

    def __call__(self) -> None:
        st = self._fn(*self._args)
        if st != PKV_OK:
            raise PagedKVError(self.name, st)


def prepare_paged_decode_attention(query, k_cache, v_cache, block_tables, context_lens,
                                   max_context_len, scale, kv_scale=1.0, workspace=None,
                                   out=None, stream=None, prefix=False) -> PreparedCall:
    """pkv_paged_decode_attention (or the prefix-aware entry) as a PreparedCall."""
    args, workspace, out = _marshal().decode(query, k_cache, v_cache, block_tables, context_lens,
                                             max_context_len, scale, kv_scale, workspace, out,
                                             stream, prefix, True)
    fn = "pkv_paged_decode_attention_prefix" if prefix else "pkv_paged_decode_attention"
    return PreparedCall(fn, args, (query, k_cache, v_cache, block_tables, context_lens,
                                   workspace, out))


def pkv_multi_query_workspace_bytes(num_seqs: int) -> int:
    return int(load().pkv_multi_query_workspace_bytes(int(num_seqs)))


def pkv_paged_multi_query_attention(query: torch.Tensor, k_cache: torch.Tensor,
                                    v_cache: torch.Tensor, block_tables: torch.Tensor,
                                    context_lens: torch.Tensor, query_start: torch.Tensor,
                                    max_context_len: int, scale: float, kv_scale: float = 1.0,
                                    workspace: torch.Tensor | None = None,
                                    out: torch.Tensor | None = None,
                                    stream=None) -> torch.Tensor:
    """Causal attention of several query tokens per sequence over the paged cache.

    query [total_q, Hq, d]; query_start int32 [S + 1] (rows of sequence s are
    query_start[s] .. query_start[s+1]-1; query_start[S] = total_q);
    context_lens int32 [S] counts the cached tokens including the queries'
    own (the last n_s).  Row i of sequence s attends to tokens
    0 .. context_lens[s] - n_s + i.
    """
    return _multi_query("pkv_paged_multi_query_attention", query, k_cache, v_cache,
                        block_tables, context_lens, query_start, None, max_context_len, scale,
                        kv_scale, workspace, out, stream)


def pkv_paged_tree_attention(query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                             block_tables: torch.Tensor, context_lens: torch.Tensor,
                             query_start: torch.Tensor, tree_mask: torch.Tensor,
                             max_context_len: int, scale: float, kv_scale: float = 1.0,
                             workspace: torch.Tensor | None = None,
                             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Verification of draft-token trees: as pkv_paged_multi_query_attention, but the
    n_s <= 64 queries of sequence s are a tree laid out parents first, and query i sees
    the prior context, itself and each tree token j < i whose bit j is set in
    tree_mask[query_start[s] + i] (int64 / uint64 bits, [total_q])."""
    if tree_mask.dtype not in (torch.int64, torch.uint64) or tree_mask.dim() != 1 or \
            int(tree_mask.shape[0]) != int(query.shape[0]):
        raise ValueError("tree_mask must be 64-bit [total_q]")
    _cuda(tree_mask, "tree_mask")
    return _multi_query("pkv_paged_tree_attention", query, k_cache, v_cache, block_tables,
                        context_lens, query_start, tree_mask, max_context_len, scale, kv_scale,
                        workspace, out, stream)


def _multi_query(name, query, k_cache, v_cache, block_tables, context_lens, query_start,
                 tree_mask, max_context_len, scale, kv_scale, workspace, out, stream):
    total_q, Hq, d = query.shape
    NB, Hkv, B, d2 = k_cache.shape
    S = int(context_lens.shape[0])
    if d2 != d or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("cache shapes must be [num_blocks, num_kv_heads, block_size, head_dim]")
    _one_type(k_cache, v_cache)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32 or \
            query_start.dtype != torch.int32:
        raise ValueError("block_tables, context_lens and query_start must be int32")
    if int(query_start.shape[0]) != S + 1:
        raise ValueError("query_start must have num_seqs + 1 entries")
    for t, n in ((query, "query"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (block_tables, "block_tables"), (context_lens, "context_lens"),
                 (query_start, "query_start")):
        _cuda(t, n)
    need = pkv_multi_query_workspace_bytes(S)
    if workspace is None:
        workspace = _fresh(query, stream, max(need, 256))
    if out is None:
        out = _fresh(query, stream)
    _cuda(out, "out")
    _cuda(workspace, "workspace")
    head = [query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
            context_lens.data_ptr(), query_start.data_ptr()]
    if tree_mask is not None:
        head.append(tree_mask.data_ptr())
    st = getattr(load(), name)(
        *head, S, total_q, Hq, Hkv, d, B, NB,
        block_tables.shape[1], int(max_context_len), float(scale), dtype_code(query),
        dtype_code(k_cache), float(kv_scale), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), out.data_ptr(), _stream_ptr(stream))
    _check(name, st)
    return out


def pkv_chunk_workspace_bytes(num_seqs: int, total_q: int, num_q_heads: int, num_kv_heads: int,
                              head_dim: int, max_context_len: int) -> int:
    return int(load().pkv_chunk_workspace_bytes(num_seqs, total_q, num_q_heads, num_kv_heads, head_dim,
                                                max_context_len))


def pkv_paged_chunk_attention(query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                              block_tables: torch.Tensor, context_lens: torch.Tensor,
                              query_start: torch.Tensor, max_context_len: int, scale: float,
                              window: int | None = None, sinks: int = 0, kv_scale: float = 1.0,
                              workspace: torch.Tensor | None = None,
                              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of each sequence's new tokens over its cache of 16 bits, FP8 or 4 bits.

    query [total_q, Hq, d] (float16 or bfloat16); rows query_start[s] .. query_start[s + 1] - 1
    (int32 [S + 1]) are the last of sequence s's context_lens[s] cached tokens.  The token at
    position p sees the tokens t <= p, under a ``window`` those with t > p - window and t < sinks;
    table entries of blocks that no row of a sequence sees are never read.  Caches as in
    pkv_paged_decode_attention, head_dim 64 or 128, up to 128 query heads a kv head.
    ``workspace`` (uint8, >= pkv_chunk_workspace_bytes) is allocated if None; rows behind the last
    sequence are left as they were (in an ``out`` allocated here: uninitialised).
    """
    return (_calls or _marshal()).chunk(query, k_cache, v_cache, block_tables, context_lens, query_start,
                                        max_context_len, scale, window, sinks, kv_scale, workspace, out,
                                        stream)


NOALLOC_SCRATCH_BYTES = 16 << 20   # PKV_NOALLOC_SCRATCH_BYTES


def pkv_paged_decode_attention_noalloc(query: torch.Tensor, k_cache: torch.Tensor,
                                       v_cache: torch.Tensor, block_tables: torch.Tensor,
                                       context_lens: torch.Tensor, max_context_len: int,
                                       scale: float, kv_scale: float = 1.0,
                                       out: torch.Tensor | None = None,
                                       stream=None) -> torch.Tensor:
    """Decode with the library's static device scratch instead of a workspace.

    For callers that cannot allocate device memory while they decode.  Fails
    with PKV_ERR_WORKSPACE when the sizes need more than 16 MiB of scratch.
    Calls that overlap on the GPU race on the shared scratch: keep them on
    one stream.  (``out`` is allocated here only when not given.)
    """
    S, Hq, d = query.shape
    NB, Hkv, B, _ = k_cache.shape
    kc, d2 = _cache_type(k_cache)
    if kc == PKV_FP4_E2M1 and (d2 != d or v_cache.shape != k_cache.shape or
                               v_cache.dtype != k_cache.dtype):
        raise ValueError("4-bit caches must have fp4_cache_shape(...) of query's head_dim")
    _one_type(k_cache, v_cache)
    for t, n in ((query, "query"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (block_tables, "block_tables"), (context_lens, "context_lens")):
        _cuda(t, n)
    if out is None:
        out = _fresh(query, stream)
    _cuda(out, "out")
    st = load().pkv_paged_decode_attention_noalloc(
        query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        context_lens.data_ptr(), S, Hq, Hkv, d, B, NB, block_tables.shape[1],
        int(max_context_len), float(scale), dtype_code(query), kc,
        float(kv_scale), out.data_ptr(), _stream_ptr(stream))
    _check("pkv_paged_decode_attention_noalloc", st)
    return out


def pkv_reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                          kv_scale: float = 1.0, stream=None) -> None:
    """k_cache[slot // B, h, slot % B] = key[t, h] (e4m3(x / kv_scale) for FP8 caches; codes
    and scales for 4-bit caches, uint8 of fp4_cache_shape).  key and value have one element type,
    and the two caches one; rows that are copied may have two, each its own cache's."""
    (_calls or _marshal()).write(key, value, k_cache, v_cache, slot_mapping, kv_scale,
                                 stream, False)


def prepare_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, kv_scale=1.0,
                              stream=None) -> PreparedCall:
    """pkv_reshape_and_cache as a PreparedCall."""
    args = _marshal().write(key, value, k_cache, v_cache, slot_mapping, kv_scale,
                            stream, True)
    return PreparedCall("pkv_reshape_and_cache", args,
                        (key, value, k_cache, v_cache, slot_mapping))


def pkv_gather_cache(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                     row_start: torch.Tensor, total_rows: int, out_dtype: torch.dtype,
                     kv_scale: float = 1.0, token_start: torch.Tensor | None = None,
                     key_out: torch.Tensor | None = None, value_out: torch.Tensor | None = None,
                     stream=None) -> tuple:
    """Read cached tokens back: (key, value) [total_rows, Hkv, d] of ``out_dtype``.

    Rows row_start[s] .. row_start[s + 1] - 1 (int32 [S + 1]) are the tokens of sequence s
    from token_start[s] (int32 [S]; 0 if None) on, found through block_tables int32
    [S, max_blocks].  16- and 32-bit caches are copied (``out_dtype`` is theirs); FP8 and
    4-bit ones become values in any of float32, float16 and bfloat16.  Rows outside every
    sequence's range are left as they were (in outputs allocated here: uninitialised).
    Two outputs allocated here share one storage: either keeps the memory of both.
    """
    return (_calls or _marshal()).gather(k_cache, v_cache, block_tables, row_start, total_rows,
                                         out_dtype, kv_scale, token_start, key_out, value_out, stream)


# ---------------------------------------------------------- norm + rotary --

def pkv_qk_norm_rope(query: torch.Tensor, key: torch.Tensor, cos_sin: torch.Tensor,
                     positions: torch.Tensor, q_weight: torch.Tensor | None = None,
                     k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                     interleaved: bool = False, q_out: torch.Tensor | None = None,
                     k_out: torch.Tensor | None = None, stream=None) -> tuple:
    """Per-head RMS norm (where a weight is given) and rotary embedding: (q_out, k_out).

    query [T, Hq, d] and key [T, Hkv, d] may be views of one projection's rows (heads
    contiguous, any token stride that is a multiple of 16 bytes); weights [d] of their type
    or float32; cos_sin float32 [max_position, rot_dim] holds each position's cosines, then
    sines; positions int64 [T].  ``interleaved`` rotates dims (2i, 2i + 1) instead of
    (i, i + rot_dim / 2).  q_out / k_out may be query / key themselves (in place).
    Two outputs allocated here share one storage: either keeps the memory of both.
    """
    return (_calls or _marshal()).norm_rope(query, key, cos_sin, positions, q_weight, k_weight,
                                            eps, interleaved, q_out, k_out, stream)


def pkv_qk_norm_rope_and_cache(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                               cos_sin: torch.Tensor, positions: torch.Tensor,
                               k_cache: torch.Tensor, v_cache: torch.Tensor,
                               slot_mapping: torch.Tensor, q_weight: torch.Tensor | None = None,
                               k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                               interleaved: bool = False, kv_scale: float = 1.0,
                               q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pkv_qk_norm_rope whose keys, with ``value`` [T, Hkv, d], go into the paged cache at
    slot_mapping (int64 [T], negative: not written); returns q_out.  The cache, of any type,
    holds the same bits as after pkv_qk_norm_rope and pkv_reshape_and_cache of its keys.  (Into
    FP8 and 4 bits, those two are faster for prompts: 16,384 tokens 72 us against 121.)"""
    return (_calls or _marshal()).norm_rope_write(
        query, key, value, cos_sin, positions, k_cache, v_cache, slot_mapping, q_weight, k_weight,
        eps, interleaved, kv_scale, q_out, stream)


def validate_pairs(pairs: np.ndarray, num_blocks: int) -> None:
    """Host check of the copy_blocks contract: ids in the pool, distinct dsts, no dst is a src."""
    pairs = np.asarray(pairs).reshape(-1, 2)
    if pairs.size and (pairs.min() < 0 or pairs.max() >= num_blocks):
        raise ValueError("copy_blocks: block id outside the pool")
    dst = pairs[:, 1]
    if len(set(dst.tolist())) != len(dst):
        raise ValueError("copy_blocks: a destination block repeats")
    if set(dst.tolist()) & set(pairs[:, 0].tolist()):
        raise ValueError("copy_blocks: a destination block is also a source")


def _copy_args(k_cache, v_cache, src_dst_pairs, stream):
    NB, Hkv, B, _ = k_cache.shape
    kc, d = _cache_type(k_cache)
    _cuda(k_cache, "k_cache")
    _cuda(v_cache, "v_cache")
    if isinstance(src_dst_pairs, torch.Tensor) and src_dst_pairs.is_cuda:
        pairs = src_dst_pairs
    else:
        host = np.ascontiguousarray(np.asarray(src_dst_pairs, dtype=np.int32).reshape(-1, 2))
        validate_pairs(host, NB)
        pairs = torch.from_numpy(host).to(k_cache.device)
        if stream is not None:     # dropped before the call's stream has read it
            pairs.record_stream(_torch_stream(stream))
    if pairs.dtype != torch.int32:
        raise ValueError("src_dst_pairs must be int32")
    n = pairs.numel() // 2
    return (k_cache.data_ptr(), v_cache.data_ptr(), pairs.data_ptr() if n else None, n, Hkv, d,
            B, NB, kc, _stream_ptr(stream)), pairs


def pkv_copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, src_dst_pairs,
                    stream=None) -> None:
    """Copy physical blocks src -> dst of both caches for every (src, dst) pair.

    ``src_dst_pairs``: int32 [n, 2].  A host array/tensor is validated and
    copied to the device; a CUDA tensor is used as is (the caller has
    validated it).
    """
    args, _ = _copy_args(k_cache, v_cache, src_dst_pairs, stream)
    _check("pkv_copy_blocks", load().pkv_copy_blocks(*args))


def prepare_copy_blocks(k_cache, v_cache, src_dst_pairs, stream=None) -> PreparedCall:
    """pkv_copy_blocks as a PreparedCall (device pairs are used as they are then)."""
    args, pairs = _copy_args(k_cache, v_cache, src_dst_pairs, stream)
    return PreparedCall("pkv_copy_blocks", args, (k_cache, v_cache, pairs))


def pkv_swap_blocks(src_k: torch.Tensor, src_v: torch.Tensor, dst_k: torch.Tensor,
                    dst_v: torch.Tensor, src_dst_pairs, stream=None) -> None:
    """Copy blocks between two pools (device or pinned host): dst[p[1]] = src[p[0]].

    Pools are [blocks, kv heads, B, d]; a host pool must be pinned
    (``tensor.pin_memory()``).  Host pairs are validated and staged in a pinned
    buffer; a CUDA or pinned tensor is used as is.
    """
    NBs, Hkv, B, row = src_k.shape
    kc, d = _cache_type(src_k)
    NBd = dst_k.shape[0]
    if tuple(dst_k.shape[1:]) != (Hkv, B, row) or src_v.shape != src_k.shape or \
            dst_v.shape != dst_k.shape:
        raise ValueError("pools must be [blocks, kv heads, B, d] with matching rows")
    for t, n in ((src_k, "src_k"), (src_v, "src_v"), (dst_k, "dst_k"), (dst_v, "dst_v")):
        if not t.is_contiguous() or not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{n} must be a contiguous CUDA or pinned host tensor")
    if isinstance(src_dst_pairs, torch.Tensor) and (src_dst_pairs.is_cuda or
                                                    src_dst_pairs.is_pinned()):
        pairs = src_dst_pairs
    else:
        host = np.ascontiguousarray(np.asarray(src_dst_pairs, dtype=np.int32).reshape(-1, 2))
        if host.size and (host[:, 0].min() < 0 or host[:, 0].max() >= NBs or
                          host[:, 1].min() < 0 or host[:, 1].max() >= NBd):
            raise ValueError("swap_blocks: block id outside its pool")
        if len(set(host[:, 1].tolist())) != len(host):
            raise ValueError("swap_blocks: a destination block repeats")
        pairs = torch.from_numpy(host).pin_memory()
    n = pairs.numel() // 2
    st = load().pkv_swap_blocks(src_k.data_ptr(), src_v.data_ptr(), NBs, dst_k.data_ptr(),
                                dst_v.data_ptr(), NBd, pairs.data_ptr() if n else None, n, Hkv,
                                d, B, kc, _stream_ptr(stream))
    _check("pkv_swap_blocks", st)
    if pairs is not src_dst_pairs and n:
        # the launch reads the staged pairs asynchronously: keep them alive until it ran
        (stream or torch.cuda.current_stream()).synchronize()


def pkv_get_device_status() -> int:
    """Read and clear the current device's status word (PKV_DEV_* bits). Synchronous."""
    v = ctypes.c_uint(0)
    _check("pkv_get_device_status", load().pkv_get_device_status(ctypes.byref(v)))
    return int(v.value)


def pkv_selftest_wait_bound(stream=None) -> None:
    """Launch the wait self-test: a kernel whose pipeline wait never completes gives up
    after the waits' bound (2 s) and sets DEV_WAIT_TIMEOUT in the device status word."""
    _check("pkv_selftest_wait_bound", load().pkv_selftest_wait_bound(_stream_ptr(stream)))


def pkv_status_string(status: int) -> str:
    return status_text(status)


def pkv_version() -> int:
    return int(load().pkv_version())


# ----------------------------------------------------------- block manager --

class BlockManager:
    """The library's host block manager (C ABI pkv_bm_*): free list, reference
    counts, block tables, slots and copy-on-write pairs for the device kernels."""

    def __init__(self, num_blocks: int, block_size: int, free_order=None):
        lib = load()
        self.block_size = block_size
        self.num_blocks = num_blocks
        if free_order is None:
            h = lib.pkv_bm_create(num_blocks, block_size, None, 0)
        else:
            order = np.ascontiguousarray(free_order, dtype=np.int32)
            h = lib.pkv_bm_create(num_blocks, block_size, order.ctypes.data, int(order.size))
        if not h:
            raise ValueError("pkv_bm_create: bad arguments")
        self._h = ctypes.c_void_p(h)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.pkv_bm_destroy(h)
            self._h = None

    @property
    def num_free(self) -> int:
        return int(load().pkv_bm_num_free(self._h))

    def refcount(self, block: int) -> int:
        return int(load().pkv_bm_refcount(self._h, int(block)))

    def add_sequence(self, seq_id: int, num_tokens: int) -> None:
        _check("pkv_bm_add_sequence", load().pkv_bm_add_sequence(self._h, seq_id, num_tokens))

    def fork(self, parent: int, child: int) -> None:
        _check("pkv_bm_fork", load().pkv_bm_fork(self._h, parent, child))

    def append_slot(self, seq_id: int):
        """(slot, (src, dst) copy-on-write pair or None) of the sequence's next token."""
        slot, src, dst = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
        _check("pkv_bm_append_slot", load().pkv_bm_append_slot(
            self._h, seq_id, ctypes.byref(slot), ctypes.byref(src), ctypes.byref(dst)))
        return int(slot.value), (None if src.value < 0 else (int(src.value), int(dst.value)))

    def free_sequence(self, seq_id: int) -> None:
        _check("pkv_bm_free_sequence", load().pkv_bm_free_sequence(self._h, seq_id))

    def sequence(self, seq_id: int):
        """(block table as a list, number of tokens)."""
        nb, nt = ctypes.c_int(), ctypes.c_int64()
        _check("pkv_bm_sequence", load().pkv_bm_sequence(self._h, seq_id, None, 0,
                                                          ctypes.byref(nb), ctypes.byref(nt)))
        table = np.zeros(max(1, nb.value), dtype=np.int32)
        _check("pkv_bm_sequence", load().pkv_bm_sequence(
            self._h, seq_id, table.ctypes.data, int(table.size), ctypes.byref(nb),
            ctypes.byref(nt)))
        return table[:nb.value].tolist(), int(nt.value)

    def prepare_step(self, seq_ids, max_blocks: int):
        """Append one token to each sequence: (slot_mapping int64[n], cow_pairs int32[k, 2],
        block_tables int32[n, max_blocks], context_lens int32[n])."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        n = int(ids.size)
        slots = np.zeros(n, np.int64)
        pairs = np.zeros((max(n, 1), 2), np.int32)
        tables = np.zeros((max(n, 1), max_blocks), np.int32)
        ctx = np.zeros(max(n, 1), np.int32)
        ncow = ctypes.c_int(0)
        _check("pkv_bm_prepare_step", load().pkv_bm_prepare_step(
            self._h, ids.ctypes.data, n, slots.ctypes.data, pairs.ctypes.data,
            ctypes.byref(ncow), tables.ctypes.data, max_blocks, ctx.ctypes.data))
        return slots, pairs[:ncow.value].copy(), tables[:n], ctx[:n]
