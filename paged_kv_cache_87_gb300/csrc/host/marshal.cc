// marshal.cc -- torch tensors into C-ABI calls (include/pagedkv.h), for binding.py.
//
// The checks of shapes, types and strides, the outputs' and the workspace's allocation and the
// call itself, in one extension function each.  They were Python: on the host of a GB300 an
// attribute of a tensor costs 0.1 us there and a call 15 - 25 us in all, five times what the
// kernels of a decode step take; here the host's part is 2 - 3.5 us a call in a loop of nothing else
// (a program that looks its tensors up between the calls: 4 - 6 us), most of it the launch.
//
// Arguments are positional (binding.py has the signatures and their documentation).  A wrong
// tensor raises ValueError, an element type that the library does not know KeyError, and a
// pkv_status that is not PKV_OK the class that set_error() was given, with (function, status).
// No C++ exception leaves: torch's become their Python classes.  The interpreter's lock is let go
// while memory is taken and while the library is called: a full launch queue waits for the device,
// and what the device waits for may be a callback that needs the lock.
#include <Python.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pagedkv.h"

namespace {

PyObject* g_error = nullptr;   // PagedKVError

struct Refused {};             // a Python exception is set

[[noreturn]] void refuse(PyObject* type, const char* text) {
    PyErr_SetString(type, text);
    throw Refused{};
}

void need(bool ok, const char* text) {
    if (!ok) refuse(PyExc_ValueError, text);
}

const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "a torch.Tensor is needed");
    return THPVariable_Unpack(o);
}

thread_local int g_device = -1;   // the current device, once an entry has asked for it

// The library works on the current device (its pointers, its stream, its status word).
void here(const at::Tensor& t) {
    if (g_device < 0) g_device = c10::cuda::current_device();
    need(t.get_device() == g_device, "tensors must be on the current CUDA device");
}

const at::Tensor& contiguous(PyObject* o, const char* text) {
    const at::Tensor& t = tensor(o);
    need(t.is_cuda() && t.is_contiguous(), text);
    here(t);
    return t;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}

// int(o), within 32 bits
int int32(PyObject* o, const char* text) {
    PyObject* i = PyNumber_Long(o);
    if (!i) throw Refused{};
    int over = 0;
    long long v = PyLong_AsLongLongAndOverflow(i, &over);
    Py_DECREF(i);
    if (over) v = INT64_MAX;
    need(v >= INT32_MIN && v <= INT32_MAX, text);
    return (int)v;
}

int size32(int64_t v) {
    need(v <= INT32_MAX, "a dimension does not fit in 32 bits");
    return (int)v;
}

pkv_dtype code_of(at::ScalarType t) {
    switch (t) {
    case at::kFloat: return PKV_F32;
    case at::kHalf: return PKV_F16;
    case at::kBFloat16: return PKV_BF16;
    case at::kFloat8_e4m3fn:
    case at::kByte: return PKV_FP8_E4M3;
    default: refuse(PyExc_KeyError, "an element type that the library does not know");
    }
}

// Whether two tensors hold the same element type (FP8 comes as float8_e4m3fn or as uint8).
bool one_type(const at::Tensor& a, const at::Tensor& b) {
    auto fp8 = [](at::ScalarType t) { return t == at::kFloat8_e4m3fn || t == at::kByte; };
    return a.scalar_type() == b.scalar_type() || (fp8(a.scalar_type()) && fp8(b.scalar_type()));
}

// A cache [NB, Hkv, B, row]: uint8 rows of 36 or 72 bytes are 4-bit codes with their scales.
struct Cache {
    int blocks, heads, block, d;
    pkv_dtype type;
};

Cache cache_of(const at::Tensor& t) {
    need(t.dim() == 4, "caches must be [num_blocks, num_kv_heads, block_size, head_dim]");
    const auto s = t.sizes();
    Cache c{size32(s[0]), size32(s[1]), size32(s[2]), size32(s[3]), code_of(t.scalar_type())};
    if (t.scalar_type() == at::kByte && (s[3] == 36 || s[3] == 72)) {
        c.type = PKV_FP4_E2M1;
        c.d = s[3] == 36 ? 64 : 128;
    }
    return c;
}

void check(const char* fn, pkv_status st) {
    if (st == PKV_OK) return;
    PyObject* e = g_error ? PyObject_CallFunction(g_error, "si", fn, (int)st) : nullptr;
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_Format(PyExc_RuntimeError, "%s failed: status %d", fn, (int)st);
    }
    throw Refused{};
}

// A torch.cuda.Stream's handle; None is the current stream of the current device.
pkv_stream_t stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Refused{};
    const long long v = PyLong_AsLongLong(h);
    Py_DECREF(h);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return reinterpret_cast<pkv_stream_t>(v);
}

struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// Calls f without the interpreter's lock; its status is checked with it.
template <typename F>
void call(const char* fn, F f) {
    pkv_status st;
    {
        Unlocked u;
        st = f();
    }
    check(fn, st);
}

// A new tensor for a call on `stream`, on the current device.  Its memory comes from what torch's
// allocator keeps for `stream`: a block that the current stream has dropped may still have that
// stream's work in flight, which `stream` does not wait for.  It is not given out again before
// `stream`, and the current stream, where the caller reads it, have done what they hold when it is
// dropped.  (Through at::empty, with its dispatch, a norm of one token took the host 4.1 us
// in such a loop instead of 3.5.)
at::Tensor fresh(at::IntArrayRef shape, const at::TensorOptions& options, pkv_stream_t stream) {
    int64_t n = 1;
    for (int64_t v : shape) n *= v;
    const caffe2::TypeMeta type = options.dtype();
    const size_t bytes = (size_t)n * type.itemsize();
    c10::Allocator* pool = c10::cuda::CUDACachingAllocator::get();
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream();
    const bool other = stream != current.stream();
    c10::DataPtr memory;
    if (other) {
        const c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(stream, current.device_index()));
        memory = pool->allocate(bytes);
    } else {
        memory = pool->allocate(bytes);
    }
    at::Tensor t(c10::make_intrusive<c10::TensorImpl>(
        c10::Storage(c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes,
                                                           std::move(memory), pool, true)),
        c10::DispatchKeySet(c10::DispatchKey::CUDA), type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    if (other && t.numel() != 0) t.record_stream(current.unwrap());
    return t;
}

// Two new tensors [rows, heads, d], one behind the other in one allocation, which they share: either
// keeps the memory of both (a second one is a fifth of what such a call costs the host: norm of one
// token 5.2 us with two, 4.2 with one).
void fresh_pair(int64_t rows, int64_t heads0, int64_t heads1, int64_t d, const at::TensorOptions& options,
                pkv_stream_t stream, at::Tensor* first, at::Tensor* second) {
    *first = fresh({rows * (heads0 + heads1) * d}, options, stream);
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(first->storage()), first->key_set(),
                                                     first->dtype());
    impl->set_storage_offset(rows * heads0 * d);
    impl->set_sizes_contiguous({rows, heads1, d});
    *second = at::Tensor(std::move(impl));
    first->unsafeGetTensorImpl()->set_sizes_contiguous({rows, heads0, d});
}

void count(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) refuse(PyExc_TypeError, "wrong number of arguments");
}

// The token stride of a CUDA tensor [T, heads, d] whose tokens' heads are contiguous.
int64_t head_rows(const at::Tensor& t, int64_t heads, int64_t d) {
    const auto s = t.strides();
    need(t.is_cuda() && s[2] == 1 && (heads == 1 || s[1] == d),
         "rows must be CUDA tensors [T, heads, d] with their heads contiguous");
    here(t);
    return t.size(0) > 1 ? s[0] : heads * d;
}

// The exception being handled, as a Python one.
PyObject* translated() {
    HANDLE_TH_ERRORS
    throw;
    END_HANDLE_TH_ERRORS
}

#define PKV_ENTRY(name)                                                       \
    PyObject* name##_body(PyObject* const* a, Py_ssize_t n);                  \
    PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {             \
        g_device = -1;                                                        \
        try {                                                                 \
            return name##_body(a, n);                                         \
        } catch (const Refused&) {                                            \
            return nullptr;                                                   \
        } catch (...) {                                                       \
            return translated();                                              \
        }                                                                     \
    }                                                                         \
    PyObject* name##_body(PyObject* const* a, Py_ssize_t n)

// decode(query, k_cache, v_cache, block_tables, context_lens, max_context_len, scale, kv_scale,
//        workspace, out, stream, prefix, prepare): out; with `prepare` nothing is launched and the
// result is (the C call's arguments, workspace, out).
// With a window (decode_window) two arguments more follow: window, sinks.
PyObject* decode_call(PyObject* const* a, bool windowed) {
    const char* plain = "query, caches, tables and lengths must be contiguous CUDA tensors";
    const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]), &v = tensor(a[2]), &bt = tensor(a[3]),
                     &cl = tensor(a[4]);
    need(q.dim() == 3 && bt.dim() == 2, "query must be [S, Hq, d], block_tables [S, max_blocks]");
    const Cache c = cache_of(k);
    need(c.d == q.size(2) && v.sizes() == k.sizes(),
         "cache shapes must be [num_blocks, num_kv_heads, block_size, head_dim]");
    need(one_type(k, v) && (c.type != PKV_FP4_E2M1 || v.scalar_type() == k.scalar_type()),
         "k_cache and v_cache must have one element type");
    need(bt.scalar_type() == at::kInt && cl.scalar_type() == at::kInt,
         "block_tables and context_lens must be int32");
    for (int i = 0; i < 5; ++i) contiguous(a[i], plain);
    const int S = size32(q.size(0)), Hq = size32(q.size(1)), width = size32(bt.size(1));
    need(bt.size(0) >= S && cl.numel() >= S, "block_tables and context_lens must have a row a query");
    const int max_ctx = int32(a[5], "max_context_len does not fit in 32 bits");
    const float scale = (float)number(a[6]), kv_scale = (float)number(a[7]);
    const pkv_stream_t stream = stream_of(a[10]);
    at::Tensor ws, out;
    if (a[8] != Py_None) ws = contiguous(a[8], "workspace must be a contiguous CUDA tensor");
    if (a[9] != Py_None) {
        out = contiguous(a[9], "out must be a contiguous CUDA tensor");
        need(out.nbytes() >= q.nbytes() && (out.scalar_type() == q.scalar_type() ||
                                            c10::isIntegralType(out.scalar_type(), false)),
             "out must have query's size and type, or be that many bytes in integers");
    }
    const bool prefix = truth(a[11]);
    const int window = windowed ? int32(a[13], "window does not fit in 32 bits") : 0;
    const int sinks = windowed ? int32(a[14], "sinks does not fit in 32 bits") : 0;
    const pkv_dtype qt = code_of(q.scalar_type());
    const bool prepare = truth(a[12]);
    size_t ws_bytes = 0;
    auto take = [&] {
        if (!ws.defined()) {
            const size_t bytes =
                windowed ? pkv_decode_window_workspace_bytes(S, Hq, c.heads, c.d, c.block, max_ctx, window,
                                                             sinks, qt, c.type)
                         : pkv_decode_workspace_bytes(S, Hq, c.heads, c.d, c.block, max_ctx, c.type);
            if (bytes || !windowed)
                ws = fresh({(int64_t)(bytes < 256 ? 256 : bytes)}, q.options().dtype(at::kByte), stream);
        }
        if (!out.defined()) out = fresh(q.sizes(), q.options(), stream);
        if (ws.defined()) ws_bytes = (size_t)ws.numel() * ws.element_size();
    };
    if (prepare) {
        take();
        return Py_BuildValue(
            "((KKKKKiiiiiiiidiidKnKK)NN)", (unsigned long long)q.data_ptr(),
            (unsigned long long)k.data_ptr(), (unsigned long long)v.data_ptr(),
            (unsigned long long)bt.data_ptr(), (unsigned long long)cl.data_ptr(), S, Hq, c.heads,
            c.d, c.block, c.blocks, width, max_ctx, (double)scale, (int)qt, (int)c.type,
            (double)kv_scale, (unsigned long long)ws.data_ptr(), (Py_ssize_t)ws_bytes,
            (unsigned long long)out.data_ptr(), (unsigned long long)stream,
            THPVariable_Wrap(ws), THPVariable_Wrap(out));
    }
    if (windowed) {
        call("pkv_paged_decode_attention_window", [&] {
            take();
            return pkv_paged_decode_attention_window(
                q.data_ptr(), k.data_ptr(), v.data_ptr(), static_cast<const int32_t*>(bt.data_ptr()),
                static_cast<const int32_t*>(cl.data_ptr()), S, Hq, c.heads, c.d, c.block, c.blocks, width,
                max_ctx, window, sinks, scale, qt, c.type, kv_scale, ws.defined() ? ws.data_ptr() : nullptr,
                ws_bytes, out.data_ptr(), stream);
        });
        return THPVariable_Wrap(std::move(out));
    }
    auto* fn = prefix ? pkv_paged_decode_attention_prefix : pkv_paged_decode_attention;
    call(prefix ? "pkv_paged_decode_attention_prefix" : "pkv_paged_decode_attention", [&] {
        take();
        return fn(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                  static_cast<const int32_t*>(bt.data_ptr()),
                  static_cast<const int32_t*>(cl.data_ptr()), S, Hq, c.heads, c.d, c.block,
                  c.blocks, width, max_ctx, scale, qt, c.type, kv_scale, ws.data_ptr(), ws_bytes,
                  out.data_ptr(), stream);
    });
    return THPVariable_Wrap(std::move(out));
}

PKV_ENTRY(decode) {
    count(n, 13);
    return decode_call(a, false);
}

// decode_window(the arguments of decode, window, sinks): out (nothing is prepared)
PKV_ENTRY(decode_window) {
    count(n, 15);
    need(!truth(a[12]) && !truth(a[11]), "a windowed decode has neither a prefix form nor a prepared one");
    return decode_call(a, true);
}

// chunk(query, k_cache, v_cache, block_tables, context_lens, query_start, max_context_len, scale, window,
//       sinks, kv_scale, workspace, out, stream): out
PKV_ENTRY(chunk) {
    count(n, 14);
    const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]), &v = tensor(a[2]), &bt = tensor(a[3]),
                     &cl = tensor(a[4]), &qs = tensor(a[5]);
    need(q.dim() == 3 && bt.dim() == 2 && cl.dim() == 1 && qs.dim() == 1,
         "query must be [total_q, Hq, d], block_tables [S, max_blocks], context_lens [S], query_start [S + 1]");
    const Cache c = cache_of(k);
    need(c.d == q.size(2) && v.sizes() == k.sizes(),
         "cache shapes must be [num_blocks, num_kv_heads, block_size, head_dim]");
    need(one_type(k, v) && (c.type != PKV_FP4_E2M1 || v.scalar_type() == k.scalar_type()),
         "k_cache and v_cache must have one element type");
    need(bt.scalar_type() == at::kInt && cl.scalar_type() == at::kInt && qs.scalar_type() == at::kInt,
         "block_tables, context_lens and query_start must be int32");
    for (int i = 0; i < 6; ++i)
        contiguous(a[i], "query, caches, tables, lengths and query_start must be contiguous CUDA tensors");
    const int S = size32(cl.size(0)), T = size32(q.size(0)), Hq = size32(q.size(1)), width = size32(bt.size(1));
    need(bt.size(0) == S && qs.size(0) == (int64_t)S + 1,
         "block_tables must have a row and query_start an entry a sequence, and one more");
    const int max_ctx = int32(a[6], "max_context_len does not fit in 32 bits");
    const float scale = (float)number(a[7]), kv_scale = (float)number(a[10]);
    const int window = a[8] == Py_None ? INT32_MAX : int32(a[8], "window does not fit in 32 bits");
    const int sinks = int32(a[9], "sinks does not fit in 32 bits");
    const pkv_stream_t stream = stream_of(a[13]);
    at::Tensor ws, out;
    if (a[11] != Py_None) ws = contiguous(a[11], "workspace must be a contiguous CUDA tensor");
    if (a[12] != Py_None) {
        out = contiguous(a[12], "out must be a contiguous CUDA tensor");
        need(out.sizes() == q.sizes() && out.scalar_type() == q.scalar_type(), "out must have query's shape and type");
    }
    const pkv_dtype qt = code_of(q.scalar_type());
    call("pkv_paged_chunk_attention", [&] {
        if (!ws.defined()) {
            const size_t bytes = pkv_chunk_workspace_bytes(S, T, Hq, c.heads, c.d, max_ctx);
            ws = fresh({(int64_t)(bytes < 256 ? 256 : bytes)}, q.options().dtype(at::kByte), stream);
        }
        if (!out.defined()) out = fresh(q.sizes(), q.options(), stream);
        return pkv_paged_chunk_attention(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), static_cast<const int32_t*>(bt.data_ptr()),
            static_cast<const int32_t*>(cl.data_ptr()), static_cast<const int32_t*>(qs.data_ptr()), S, T, Hq,
            c.heads, c.d, c.block, c.blocks, width, max_ctx, window, sinks, scale, qt, c.type, kv_scale,
            ws.data_ptr(), (size_t)ws.numel() * ws.element_size(), out.data_ptr(), stream);
    });
    return THPVariable_Wrap(std::move(out));
}

// write(key, value, k_cache, v_cache, slot_mapping, kv_scale, stream, prepare): None, or the C
// call's arguments.
PKV_ENTRY(write) {
    count(n, 8);
    const at::Tensor &key = tensor(a[0]), &value = tensor(a[1]), &k = tensor(a[2]),
                     &v = tensor(a[3]), &slots = tensor(a[4]);
    need(key.dim() == 3, "key must be [T, Hkv, d]");
    const Cache c = cache_of(k);
    need(key.size(1) == c.heads && key.size(2) == c.d && value.sizes() == key.sizes(),
         "key/value [T, Hkv, d] do not match the cache [NB, Hkv, B, d]");
    need(v.dim() == 4 && v.size(0) >= k.size(0) && v.sizes().slice(1) == k.sizes().slice(1),
         "k_cache and v_cache must have one shape (v_cache may have more blocks)");
    // rows that are copied may be of two types, each of its own cache's
    const bool copied = key.scalar_type() == k.scalar_type() && value.scalar_type() == v.scalar_type() &&
                        value.element_size() == key.element_size();
    need(copied || (one_type(k, v) && value.scalar_type() == key.scalar_type() &&
                    (c.type != PKV_FP4_E2M1 || v.scalar_type() == k.scalar_type())),
         "key and value, and the two caches, must have one element type");
    need(slots.scalar_type() == at::kLong && slots.numel() >= key.size(0),
         "slot_mapping must be int64 [T]");
    for (int i = 0; i < 5; ++i)
        contiguous(a[i], "rows, caches and slot_mapping must be contiguous CUDA tensors");
    const int T = size32(key.size(0));
    const float kv_scale = (float)number(a[5]);
    const pkv_dtype st = code_of(key.scalar_type());
    const pkv_stream_t stream = stream_of(a[6]);
    if (truth(a[7]))
        return Py_BuildValue("(KKKKKiiiiiiidK)", (unsigned long long)key.data_ptr(),
                             (unsigned long long)value.data_ptr(), (unsigned long long)k.data_ptr(),
                             (unsigned long long)v.data_ptr(), (unsigned long long)slots.data_ptr(),
                             T, c.heads, c.d, c.block, c.blocks, (int)st, (int)c.type,
                             (double)kv_scale, (unsigned long long)stream);
    call("pkv_reshape_and_cache", [&] {
        return pkv_reshape_and_cache(key.data_ptr(), value.data_ptr(), k.data_ptr(), v.data_ptr(),
                                     static_cast<const int64_t*>(slots.data_ptr()), T, c.heads, c.d,
                                     c.block, c.blocks, st, c.type, kv_scale, stream);
    });
    Py_RETURN_NONE;
}

// gather(k_cache, v_cache, block_tables, row_start, total_rows, out_dtype, kv_scale, token_start,
//        key_out, value_out, stream): (key, value)
PKV_ENTRY(gather) {
    count(n, 11);
    const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]), &bt = tensor(a[2]), &rs = tensor(a[3]);
    const Cache c = cache_of(k);
    need(v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type(),
         "k_cache and v_cache must have one shape and type");
    need(bt.dim() == 2 && bt.scalar_type() == at::kInt && rs.dim() == 1 &&
             rs.scalar_type() == at::kInt && rs.size(0) == bt.size(0) + 1,
         "block_tables must be int32 [S, max_blocks], row_start int32 [S + 1]");
    for (int i = 0; i < 4; ++i)
        contiguous(a[i], "caches, block_tables and row_start must be contiguous CUDA tensors");
    const int32_t* first = nullptr;
    if (a[7] != Py_None) {
        const at::Tensor& ts = contiguous(a[7], "token_start must be a contiguous CUDA tensor");
        need(ts.scalar_type() == at::kInt && ts.dim() == 1 && ts.size(0) == bt.size(0),
             "token_start must be int32 [S]");
        first = static_cast<const int32_t*>(ts.data_ptr());
    }
    const int rows = int32(a[4], "total_rows does not fit in 32 bits");
    need(rows >= 0, "total_rows must not be negative");
    need(THPDtype_Check(a[5]), "out_dtype must be a torch.dtype");
    const at::ScalarType type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    const pkv_dtype out_type = code_of(type);
    const int64_t shape[3] = {rows, c.heads, c.d};
    const int S = size32(bt.size(0)), width = size32(bt.size(1));
    const float kv_scale = (float)number(a[6]);
    const pkv_stream_t stream = stream_of(a[10]);
    at::Tensor out[2];
    for (int i = 0; i < 2; ++i)
        if (a[8 + i] != Py_None) {
            out[i] = contiguous(a[8 + i], "key_out and value_out must be contiguous CUDA tensors");
            need(out[i].sizes() == at::IntArrayRef(shape, 3) && out[i].scalar_type() == type,
                 "key_out and value_out must be [total_rows, Hkv, d] of out_dtype");
        }
    call("pkv_gather_cache", [&] {
        if (!out[0].defined() && !out[1].defined())
            fresh_pair(rows, c.heads, c.heads, c.d, k.options().dtype(type), stream, &out[0], &out[1]);
        for (at::Tensor& t : out)
            if (!t.defined()) t = fresh(shape, k.options().dtype(type), stream);
        return pkv_gather_cache(k.data_ptr(), v.data_ptr(),
                                static_cast<const int32_t*>(bt.data_ptr()),
                                static_cast<const int32_t*>(rs.data_ptr()), first, S, rows, c.heads,
                                c.d, c.block, c.blocks, width, c.type, kv_scale, out_type,
                                out[0].data_ptr(), out[1].data_ptr(), stream);
    });
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(out[0])), THPVariable_Wrap(std::move(out[1])));
}

// What the two norm + rotary calls share, from their first arguments.
struct NormRope {
    const at::Tensor *q, *k, *cs, *pos;
    at::Tensor q_out;
    const void *qw = nullptr, *kw = nullptr;
    pkv_dtype type, weight_type = PKV_F32;
    int T, Hq, Hkv, d, positions_known, rot_dim;
    int64_t q_stride, k_stride, out_stride;
    float eps;
    bool interleaved;
    pkv_stream_t stream;

    NormRope(PyObject* query, PyObject* key, PyObject* cos_sin, PyObject* positions, PyObject* q_w,
             PyObject* k_w, PyObject* eps_, PyObject* interleaved_, PyObject* out, PyObject* stream_) {
        q = &tensor(query);
        k = &tensor(key);
        need(q->dim() == 3 && k->dim() == 3 && q->size(0) == k->size(0) &&
                 q->size(2) == k->size(2) && q->scalar_type() == k->scalar_type(),
             "query [T, Hq, d] and key [T, Hkv, d] must agree in T, d and type");
        T = size32(q->size(0));
        Hq = size32(q->size(1));
        Hkv = size32(k->size(1));
        d = size32(q->size(2));
        type = code_of(q->scalar_type());
        cs = &contiguous(cos_sin, "cos_sin must be a contiguous CUDA tensor");
        need(cs->dim() == 2 && cs->scalar_type() == at::kFloat,
             "cos_sin must be float32 [max_position, rot_dim]");
        positions_known = size32(cs->size(0));
        rot_dim = size32(cs->size(1));
        pos = &contiguous(positions, "positions must be a contiguous CUDA tensor");
        need(pos->dim() == 1 && pos->size(0) == T && pos->scalar_type() == at::kLong,
             "positions must be int64 [T]");
        PyObject* w[2] = {q_w, k_w};
        const void** to[2] = {&qw, &kw};
        for (int i = 0; i < 2; ++i) {
            if (w[i] == Py_None) continue;
            const at::Tensor& t = contiguous(w[i], "weights must be contiguous CUDA tensors");
            need(t.dim() == 1 && t.size(0) == d, "weights must be [head_dim]");
            const pkv_dtype c = code_of(t.scalar_type());
            need(i == 0 || !qw || c == weight_type, "q_weight and k_weight must have one type");
            weight_type = c;
            *to[i] = t.data_ptr();
        }
        q_stride = head_rows(*q, Hq, d);
        k_stride = head_rows(*k, Hkv, d);
        eps = (float)number(eps_);
        interleaved = truth(interleaved_);
        stream = stream_of(stream_);
        rows_out(out, *q, Hq, &q_out, &out_stride);
    }

    // What was given as an output, checked; nothing yet where none was.
    void rows_out(PyObject* given, const at::Tensor& like, int64_t heads, at::Tensor* to, int64_t* stride) {
        *stride = heads * d;
        if (given != Py_None) {
            *to = tensor(given);
            need(to->sizes() == like.sizes() && to->scalar_type() == like.scalar_type(),
                 "q_out and k_out must have query's and key's shape and type");
            *stride = head_rows(*to, heads, d);
        }
    }
};

// norm_rope(query, key, cos_sin, positions, q_weight, k_weight, eps, interleaved, q_out, k_out,
//           stream): (q_out, k_out)
PKV_ENTRY(norm_rope) {
    count(n, 11);
    NormRope r(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[10]);
    at::Tensor k_out;
    int64_t k_out_stride;
    r.rows_out(a[9], *r.k, r.Hkv, &k_out, &k_out_stride);
    call("pkv_qk_norm_rope", [&] {
        if (!r.q_out.defined() && !k_out.defined())
            fresh_pair(r.T, r.Hq, r.Hkv, r.d, r.q->options(), r.stream, &r.q_out, &k_out);
        if (!r.q_out.defined()) r.q_out = fresh(r.q->sizes(), r.q->options(), r.stream);
        if (!k_out.defined()) k_out = fresh(r.k->sizes(), r.k->options(), r.stream);
        return pkv_qk_norm_rope(r.q->data_ptr(), r.q_stride, r.k->data_ptr(), r.k_stride, r.qw, r.kw,
                                r.weight_type, r.eps, static_cast<const float*>(r.cs->data_ptr()),
                                r.positions_known, r.rot_dim, r.interleaved,
                                static_cast<const int64_t*>(r.pos->data_ptr()), r.T, r.Hq, r.Hkv,
                                r.d, r.type, r.q_out.data_ptr(), r.out_stride, k_out.data_ptr(),
                                k_out_stride, r.stream);
    });
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(r.q_out)), THPVariable_Wrap(std::move(k_out)));
}

// norm_rope_write(query, key, value, cos_sin, positions, k_cache, v_cache, slot_mapping, q_weight,
//                 k_weight, eps, interleaved, kv_scale, q_out, stream): q_out
PKV_ENTRY(norm_rope_write) {
    count(n, 15);
    const at::Tensor &key = tensor(a[1]), &value = tensor(a[2]), &k = tensor(a[5]), &v = tensor(a[6]),
                     &slots = tensor(a[7]);
    const Cache c = cache_of(k);
    need(key.dim() == 3 && key.size(1) == c.heads && key.size(2) == c.d && v.sizes() == k.sizes() &&
             v.scalar_type() == k.scalar_type(),
         "key [T, Hkv, d] does not match the caches [NB, Hkv, B, d]");
    need(value.sizes() == key.sizes() && value.scalar_type() == key.scalar_type(),
         "value must have key's shape and type");
    need(slots.scalar_type() == at::kLong && slots.dim() == 1 && slots.size(0) == key.size(0),
         "slot_mapping must be int64 [T]");
    for (int i = 5; i < 8; ++i)
        contiguous(a[i], "caches and slot_mapping must be contiguous CUDA tensors");
    NormRope r(a[0], a[1], a[3], a[4], a[8], a[9], a[10], a[11], a[13], a[14]);
    const int64_t v_stride = head_rows(value, r.Hkv, r.d);
    const float kv_scale = (float)number(a[12]);
    call("pkv_qk_norm_rope_and_cache", [&] {
        if (!r.q_out.defined()) r.q_out = fresh(r.q->sizes(), r.q->options(), r.stream);
        return pkv_qk_norm_rope_and_cache(
            r.q->data_ptr(), r.q_stride, r.k->data_ptr(), r.k_stride, value.data_ptr(), v_stride,
            r.qw, r.kw, r.weight_type, r.eps, static_cast<const float*>(r.cs->data_ptr()),
            r.positions_known, r.rot_dim, r.interleaved,
            static_cast<const int64_t*>(r.pos->data_ptr()), r.T, r.Hq, r.Hkv, r.d, r.type,
            r.q_out.data_ptr(), r.out_stride, k.data_ptr(), v.data_ptr(),
            static_cast<const int64_t*>(slots.data_ptr()), c.block, c.blocks, c.type, kv_scale,
            r.stream);
    });
    return THPVariable_Wrap(std::move(r.q_out));
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

#define PKV_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {PKV_FAST(decode), PKV_FAST(decode_window), PKV_FAST(chunk), PKV_FAST(write), PKV_FAST(gather), PKV_FAST(norm_rope),
                           PKV_FAST(norm_rope_write), {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
    PyObject* m = PyModule_Create(&g_module);
    // the torch it was compiled for: binding.py asks, for no interface of torch's C++ stays the same
    if (m && PyModule_AddStringConstant(m, "TORCH", PKV_TORCH) < 0) Py_CLEAR(m);
    return m;
}
