// step_binding.cpp -- Python binding of the serving-step operators, argument
// marshalling only: checks tensors, allocates outputs, calls the C ABI.
//
// A serving step calls these for every layer, and at small sizes a call costs
// more on the host than on the GPU; the same checks written in Python and passed
// through ctypes took 8 to 25 us a call.  _paged.py and _latent.py hold the signatures and
// their documentation and pass every argument by position.  The C entries are
// handed over by _lib.py, which loads libkda.so.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <string>

#include "kda.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Entries {
    decltype(&kda_build_block_tables) tables;
    decltype(&kda_cache_append) append;
    decltype(&kda_paged_attention_workspace_size) attention_size;
    decltype(&kda_paged_attention) attention;
    decltype(&kda_verify_draft) verify;
    decltype(&kda_rotary) rotary;
    decltype(&kda_latent_append) latent_append;
    decltype(&kda_latent_attention_workspace_size) latent_size;
    decltype(&kda_latent_attention) latent;
    decltype(&kda_expanded_attention_workspace_size) expanded_size;
    decltype(&kda_expanded_attention) expanded;
} g_kda{};
PyObject* g_error = nullptr;                           // _lib.KDAError

struct Refused {};                                     // a Python exception is set

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Refused{};
}
[[noreturn]] void value_error(const std::string& what) { refuse(PyExc_ValueError, what); }

std::string str(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}
std::string str(ScalarType t) {
    switch (t) {
        case ScalarType::Half: return "torch.float16";
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Float: return "torch.float32";
        case ScalarType::Double: return "torch.float64";
        case ScalarType::Int: return "torch.int32";
        case ScalarType::Long: return "torch.int64";
        default: return at::toString(t);
    }
}

const Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
int64_t integer(const char* name, PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " is out of range");
    return v;
}

// a Python value's truth; asking may raise
bool truth(PyObject* o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw Refused{};
    return t != 0;
}

void check_shape(const char* name, const Tensor& t, at::IntArrayRef shape) {
    if (t.sizes() != shape) value_error(std::string(name) + " must have shape " + str(shape) + ", got " + str(t.sizes()));
}
// the C entries take sizes as int; a larger one must not be cut off
void check_size(const char* name, const Tensor& t) {
    for (const int64_t n : t.sizes())
        if (n > INT32_MAX) value_error(std::string(name) + " " + str(t.sizes()) + " has a dim past 2^31 - 1");
}
void check_kind(const char* name, const Tensor& t, int dev, ScalarType dtype) {
    if (t.scalar_type() != dtype) refuse(PyExc_TypeError, std::string(name) + " must be " + str(dtype) + ", got " + str(t.scalar_type()));
    if (!t.is_cuda() || t.get_device() != dev) value_error(std::string(name) + " must be on cuda:" + std::to_string(dev));
}
// pointer of a contiguous tensor of that dtype and shape on that device
void* need(const char* name, const Tensor& t, int dev, ScalarType dtype, at::IntArrayRef shape) {
    check_shape(name, t, shape);
    check_kind(name, t, dev, dtype);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return t.data_ptr();
}
int device_of(const char* name, const Tensor& t) {
    if (!t.is_cuda()) value_error(std::string(name) + " must be on a CUDA device");
    return t.get_device();
}
kda_dtype code_of(const Tensor& t) {
    if (t.scalar_type() == ScalarType::BFloat16) return KDA_BF16;
    if (t.scalar_type() == ScalarType::Float) return KDA_FP32;
    refuse(PyExc_TypeError, "KDA supports bfloat16 and float32, not " + str(t.scalar_type()));
}
// a [tokens, heads, d] tensor whose tokens may lie further apart than heads * d (a slice
// of a fused projection): pointer, and elements between tokens
const void* rows(const char* name, const Tensor& t, int dev, ScalarType dtype, at::IntArrayRef shape, int64_t& stride) {
    check_shape(name, t, shape);
    check_kind(name, t, dev, dtype);
    const int64_t row = shape[1] * shape[2];
    stride = row;
    if (t.is_contiguous()) return t.data_ptr();
    if ((t.stride(2) != 1 && shape[2] > 1) || (t.stride(1) != shape[2] && shape[1] > 1))
        value_error(std::string(name) + ": the heads of a token must be contiguous");
    if (shape[0] > 1 && t.stride(0) < row) value_error(std::string(name) + ": tokens must not overlap");
    stride = std::max(t.stride(0), row);
    return t.data_ptr();
}
// a [tokens, heads, d] tensor whose tokens and heads may lie at any strides: pointer and
// strides in elements (of a dim of one: as if it were packed).  Whether rows overlap is the C entry's to judge.
const void* strided(const char* name, const Tensor& t, int dev, ScalarType dtype, at::IntArrayRef shape, int64_t& token,
                    int64_t& head) {
    check_shape(name, t, shape);
    check_kind(name, t, dev, dtype);
    if (t.stride(2) != 1 && shape[2] > 1) value_error(std::string(name) + ": the channels of a head must be contiguous");
    head = shape[1] > 1 ? t.stride(1) : shape[2];
    token = shape[0] > 1 ? t.stride(0) : std::max(t.stride(1), shape[2]) * shape[1];
    return t.data_ptr();
}
double number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Refused{};
    return x;
}
// The stream of a call.  Tensors made here are that stream's own memory: the current
// stream's could still be read or written by work queued there before they were freed, and
// torch may fill new memory, which must come before the call's kernels.  What the caller gets is
// most likely used on the current stream next, so its memory is not handed out again
// before that stream is done with it either.
struct Stream {
    cudaStream_t handle;
    c10::cuda::CUDAStream current;
    Tensor make(const Tensor& like, ScalarType dtype, at::IntArrayRef shape) const {
        const auto options = like.options().dtype(dtype).requires_grad(false);
        if (handle == current.stream()) return at::empty(shape, options);
        const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(handle, current.device_index()));
        Tensor t = at::empty(shape, options);
        if (t.numel() > 0) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current);
        return t;
    }
};
Stream stream_of(PyObject* o, int dev) {
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev);
    if (o == Py_None) return {current.stream(), current};
    if (PyObject_HasAttrString(o, "device_index")) {       // a torch stream; a raw handle does not tell
        PyObject* index = PyObject_GetAttrString(o, "device_index");
        if (!index) throw Refused{};
        const long of = PyLong_AsLong(index);
        Py_DECREF(index);
        if (of == -1 && PyErr_Occurred()) throw Refused{};
        if (of != dev) value_error("stream must be on cuda:" + std::to_string(dev) + ", not cuda:" + std::to_string(of));
    }
    PyObject* handle = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Long(o);
    if (!handle) throw Refused{};
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!p && PyErr_Occurred()) throw Refused{};
    return {static_cast<cudaStream_t>(p), current};
}

// the caller's output tensor, checked, or a new one (None)
Tensor out(const char* name, PyObject* o, const Stream& s, const Tensor& like, ScalarType dtype, at::IntArrayRef shape) {
    if (o == Py_None) return s.make(like, dtype, shape);
    const Tensor& t = tensor(name, o);
    need(name, t, s.current.device_index(), dtype, shape);
    return t;
}

// Gives up the interpreter lock; an exception that passes through gets it back first.
struct Unlocked {
    PyThreadState* const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// Calls a C entry with `dev` current (the library looks up the SM count and the
// status word of the current device); raises on an error code.
template <typename F>
void call(const char* entry, int dev, F f) {
    kda_status st;
    {
        c10::cuda::OptionalCUDAGuard guard;
        if (c10::cuda::current_device() != dev) guard.set_index((c10::DeviceIndex)dev);
        const Unlocked unlocked;
        st = f();
    }
    if (st == KDA_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, entry);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused{};
}

template <typename F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, F f) {
    try {
        if (got != want) refuse(PyExc_TypeError, std::string(name) + ": wrong number of arguments");
        if (!g_error) refuse(PyExc_RuntimeError, "the KDA library is not loaded");
        return f();
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
        return nullptr;
    }
}

PyObject* tuple(std::initializer_list<Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw Refused{};
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
    return r;
}

constexpr ScalarType kI32 = ScalarType::Int, kI64 = ScalarType::Long, kF32 = ScalarType::Float;

PyObject* build_block_tables(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded("kda_build_block_tables", n_args, 12, [&] {
        const Tensor &ctx = tensor("ctx_len", a[0]), &add = tensor("new_len", a[1]), &free = tensor("free_pages", a[2]),
                     &table = tensor("block_table", a[3]);
        if (ctx.dim() != 1 || table.dim() != 2 || free.dim() != 1)
            value_error("ctx_len and free_pages must have 1 dim, block_table 2");
        check_size("ctx_len", ctx);
        check_size("free_pages", free);
        check_size("block_table", table);
        const int64_t n = ctx.size(0), blocks = table.size(1), n_free = free.size(0);
        check_shape("new_len", add, {n});
        const int64_t page = integer("page_size", a[4]), n_tokens = integer("n_tokens", a[5]);
        if (n_tokens < 0) value_error("n_tokens must not be negative");
        const int dev = device_of("ctx_len", ctx);
        void *ctx_p = need("ctx_len", ctx, dev, kI32, {n}), *add_p = need("new_len", add, dev, kI32, {n}),
             *free_p = need("free_pages", free, dev, kI32, {n_free}), *table_p = need("block_table", table, dev, kI32, {n, blocks});
        const Stream s = stream_of(a[11], dev);
        Tensor cu = out("cu_seqlens", a[6], s, ctx, kI32, {n + 1}), seq = out("seq_len", a[7], s, ctx, kI32, {n}),
               slot = out("slot_map", a[8], s, ctx, kI64, {n_tokens}), pos = out("positions", a[9], s, ctx, kI32, {n_tokens}),
               taken = out("n_taken", a[10], s, ctx, kI32, {1});
        call("kda_build_block_tables", dev, [&] {
            return g_kda.tables((const int32_t*)ctx_p, (const int32_t*)add_p, (const int32_t*)free_p, (int)n_free, (int)n,
                                (int)blocks, (int)page, (int)n_tokens, (int32_t*)table_p, (int32_t*)cu.data_ptr(),
                                (int32_t*)seq.data_ptr(), (int64_t*)slot.data_ptr(), (int32_t*)pos.data_ptr(),
                                (int32_t*)taken.data_ptr(), s.handle);
        });
        return tuple({cu, seq, slot, pos, taken});
    });
}

void check_caches(const char* entry, const Tensor& k, const Tensor& v) {
    if (k.dim() != 4 || v.sizes() != k.sizes())
        value_error(std::string(entry) + ": k_cache and v_cache must have one shape [n_pages, H_kv, page_size, d], got " +
                    str(k.sizes()) + " and " + str(v.sizes()));
    check_size("k_cache", k);
}

PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded("kda_cache_append", n_args, 6, [&] {
        const Tensor &k = tensor("k", a[0]), &v = tensor("v", a[1]), &kc = tensor("k_cache", a[2]),
                     &vc = tensor("v_cache", a[3]), &slot = tensor("slot_map", a[4]);
        check_caches("kda_cache_append", kc, vc);
        if (k.dim() != 3) value_error("k must have 3 dims, got " + std::to_string(k.dim()));
        check_size("k", k);
        const int64_t shape[3] = {k.size(0), kc.size(1), kc.size(3)};
        const kda_dtype code = code_of(kc);
        const ScalarType dt = kc.scalar_type();
        check_shape("k", k, shape);
        check_shape("v", v, shape);
        const int dev = device_of("k_cache", kc);
        int64_t ks, vs;
        const void *kp = rows("k", k, dev, dt, shape, ks), *vp = rows("v", v, dev, dt, shape, vs);
        void *kcp = need("k_cache", kc, dev, dt, kc.sizes()), *vcp = need("v_cache", vc, dev, dt, kc.sizes()),
             *sp = need("slot_map", slot, dev, kI64, {shape[0]});
        const Stream s = stream_of(a[5], dev);
        call("kda_cache_append", dev, [&] {
            return g_kda.append(kp, vp, (const int64_t*)sp, ks, vs, (int)shape[0], (int)shape[1], (int)shape[2],
                                (int)kc.size(2), (int)kc.size(0), code, kcp, vcp, s.handle);
        });
        Py_RETURN_NONE;
    });
}

PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded("kda_paged_attention", n_args, 13, [&]() -> PyObject* {
        const Tensor &q = tensor("q", a[0]), &kc = tensor("k_cache", a[1]), &vc = tensor("v_cache", a[2]),
                     &table = tensor("block_table", a[3]), &cu = tensor("cu_seqlens", a[4]), &seq = tensor("seq_len", a[5]);
        check_caches("kda_paged_attention", kc, vc);
        if (q.dim() != 3 || table.dim() != 2)
            value_error("q must have 3 dims and block_table 2, got " + std::to_string(q.dim()) + " and " + std::to_string(table.dim()));
        check_size("q", q);
        check_size("block_table", table);
        const int64_t T = q.size(0), heads = q.size(1), d = kc.size(3), kv_heads = kc.size(1), n = table.size(0),
                      blocks = table.size(1);
        if (q.size(2) != d || kv_heads == 0 || heads % kv_heads != 0)
            value_error("q " + str(q.sizes()) + " does not match caches of " + std::to_string(kv_heads) + " heads of " + std::to_string(d));
        const kda_dtype code = code_of(q);
        const ScalarType dt = q.scalar_type();
        if (cu.sizes() != at::IntArrayRef({n + 1}) || seq.sizes() != at::IntArrayRef({n}))
            value_error("cu_seqlens and seq_len must have shapes " + str(at::IntArrayRef({n + 1})) + " and " +
                        str(at::IntArrayRef({n})) + ", got " + str(cu.sizes()) + " and " + str(seq.sizes()));
        double scale = 0.0;
        if (a[6] == Py_None) {
            scale = 1.0 / std::sqrt((double)d);
        } else {
            scale = PyFloat_AsDouble(a[6]);
            if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
        }
        const int64_t window = integer("window", a[7]);
        const bool want_lse = a[9] != Py_None || truth(a[10]);
        if (a[8] != Py_None) check_shape("o", tensor("o", a[8]), q.sizes());
        if (a[9] != Py_None) check_shape("lse", tensor("lse", a[9]), {T, heads});
        const int dev = device_of("q", q);
        int64_t qs;
        const void* qp = rows("q", q, dev, dt, q.sizes(), qs);
        void *kcp = need("k_cache", kc, dev, dt, kc.sizes()), *vcp = need("v_cache", vc, dev, dt, kc.sizes()),
             *tp = need("block_table", table, dev, kI32, table.sizes()), *cup = need("cu_seqlens", cu, dev, kI32, {n + 1}),
             *sp = need("seq_len", seq, dev, kI32, {n});
        const Stream s = stream_of(a[12], dev);
        Tensor o = out("o", a[8], s, q, dt, q.sizes()), lse;
        if (want_lse) lse = out("lse", a[9], s, q, kF32, {T, heads});
        Tensor ws;
        size_t bytes;
        if (a[11] == Py_None) {
            bytes = g_kda.attention_size((int)T, (int)heads, (int)kv_heads, (int)d, code);
            ws = s.make(q, ScalarType::Byte, {(int64_t)bytes});
        } else {
            ws = tensor("workspace", a[11]);
            if (!ws.is_cuda() || ws.get_device() != dev || !ws.is_contiguous())
                value_error("workspace must be contiguous and on cuda:" + std::to_string(dev));
            bytes = (size_t)ws.numel() * ws.element_size();
        }
        call("kda_paged_attention", dev, [&] {
            return g_kda.attention(qp, kcp, vcp, (const int32_t*)tp, (const int32_t*)cup, (const int32_t*)sp, qs, (int)n,
                                   (int)T, (int)heads, (int)kv_heads, (int)d, (int)kc.size(2), (int)blocks, (int)kc.size(0),
                                   (float)scale, (int)window, code, o.data_ptr(),
                                   want_lse ? (float*)lse.data_ptr() : nullptr, ws.data_ptr(), bytes, s.handle);
        });
        if (want_lse) return tuple({o, lse});
        return THPVariable_Wrap(o);
    });
}

PyObject* verify_draft(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded("kda_verify_draft", n_args, 8, [&] {
        const Tensor &p = tensor("target", a[0]), &t = tensor("draft_tokens", a[2]), &u = tensor("uniforms", a[3]);
        const bool has_draft = a[1] != Py_None, has_len = a[4] != Py_None;
        if (p.dim() != 3 || t.dim() != 2)
            value_error("target must have 3 dims and draft_tokens 2, got " + std::to_string(p.dim()) + " and " + std::to_string(t.dim()));
        check_size("target", p);
        check_size("draft_tokens", t);
        const int64_t n = t.size(0), k = t.size(1), vocab = p.size(2);
        const int64_t p_shape[3] = {n, k + 1, vocab}, q_shape[3] = {n, k, vocab};
        if (p.sizes() != at::IntArrayRef(p_shape) || (has_draft && tensor("draft", a[1]).sizes() != at::IntArrayRef(q_shape)))
            value_error("target and draft must have shapes " + str(p_shape) + " and " + str(q_shape) + ", got " + str(p.sizes()) +
                        " and " + (has_draft ? str(tensor("draft", a[1]).sizes()) : "None"));
        check_shape("uniforms", u, {n, k + 1});
        const kda_dtype code = code_of(p);
        const ScalarType dt = p.scalar_type();
        const int dev = device_of("target", p);
        void *pp = need("target", p, dev, dt, p_shape), *qp = has_draft ? need("draft", tensor("draft", a[1]), dev, dt, q_shape) : nullptr,
             *tp = need("draft_tokens", t, dev, kI32, {n, k}), *up = need("uniforms", u, dev, kF32, {n, k + 1}),
             *lp = has_len ? need("draft_len", tensor("draft_len", a[4]), dev, kI32, {n}) : nullptr;
        const Stream s = stream_of(a[7], dev);
        Tensor tokens = out("tokens", a[5], s, p, kI32, {n, k + 1}), commit = out("commit_len", a[6], s, p, kI32, {n});
        call("kda_verify_draft", dev, [&] {
            return g_kda.verify(pp, qp, (const int32_t*)tp, (const float*)up, (const int32_t*)lp, (int)n, (int)k, (int)vocab,
                                code, (int32_t*)tokens.data_ptr(), (int32_t*)commit.data_ptr(), s.handle);
        });
        return tuple({tokens, commit});
    });
}

// the caller's workspace, checked, or a new one (None) of `bytes`; `bytes` becomes its size
Tensor scratch(PyObject* o, const Stream& s, const Tensor& like, size_t& bytes) {
    if (o == Py_None) return s.make(like, ScalarType::Byte, {(int64_t)bytes});
    const Tensor& ws = tensor("workspace", o);
    if (!ws.is_cuda() || ws.get_device() != s.current.device_index() || !ws.is_contiguous())
        value_error("workspace must be contiguous and on cuda:" + std::to_string(s.current.device_index()));
    bytes = (size_t)ws.numel() * ws.element_size();
    return ws;
}

PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded("kda_rotary", n_args, 7, [&] {
        const Tensor &x = tensor("x", a[0]), &pos = tensor("positions", a[1]), &freq = tensor("inv_freq", a[2]);
        if (x.dim() != 3 || freq.dim() != 1)
            value_error("x must have 3 dims and inv_freq 1, got " + std::to_string(x.dim()) + " and " + std::to_string(freq.dim()));
        check_size("x", x);
        const int64_t T = x.size(0), heads = x.size(1), d = x.size(2), rot = 2 * freq.size(0);
        if (rot > d) value_error("inv_freq " + str(freq.sizes()) + " has more pairs than heads of " + std::to_string(d));
        const double factor = number(a[3]);
        const bool interleaved = truth(a[4]);
        const kda_dtype code = code_of(x);
        const ScalarType dt = x.scalar_type();
        const int dev = device_of("x", x);
        int64_t xt, xh, ot, oh;
        const void *xp = strided("x", x, dev, dt, x.sizes(), xt, xh), *pp = need("positions", pos, dev, kI32, {T}),
                   *fp = need("inv_freq", freq, dev, kF32, {freq.size(0)});
        const Stream s = stream_of(a[6], dev);
        const Tensor out = a[5] == Py_None ? s.make(x, dt, x.sizes()) : tensor("out", a[5]);
        void* op = const_cast<void*>(strided("out", out, dev, dt, x.sizes(), ot, oh));
        call("kda_rotary", dev, [&] {
            return g_kda.rotary(xp, (const int32_t*)pp, (const float*)fp, xt, xh, ot, oh, (int)T, (int)heads, (int)d, (int)rot,
                                interleaved, (float)factor, code, op, s.handle);
        });
        return THPVariable_Wrap(out);
    });
}

constexpr int64_t kLatent = 512, kRope = 64, kNope = 128, kValue = 128;

void check_latent_cache(const char* entry, const Tensor& cache) {
    if (cache.dim() != 3 || cache.size(2) != kLatent + kRope)
        value_error(std::string(entry) + ": cache must have shape [n_pages, page_size, 576], got " + str(cache.sizes()));
    check_size("cache", cache);
}

// a [tokens, d] tensor whose tokens may lie further apart than d
const void* lines(const char* name, const Tensor& t, int dev, ScalarType dtype, at::IntArrayRef shape, int64_t& stride) {
    check_shape(name, t, shape);
    check_kind(name, t, dev, dtype);
    if (t.stride(1) != 1) value_error(std::string(name) + ": the channels of a token must be contiguous");
    if (shape[0] > 1 && t.stride(0) < shape[1]) value_error(std::string(name) + ": tokens must not overlap");
    stride = std::max(t.stride(0), shape[1]);
    return t.data_ptr();
}

PyObject* latent_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded("kda_latent_append", n_args, 9, [&] {
        const Tensor &c = tensor("c", a[0]), &r = tensor("k_rope", a[1]), &cache = tensor("cache", a[2]), &slot = tensor("slot_map", a[3]);
        check_latent_cache("kda_latent_append", cache);
        if (c.dim() != 2) value_error("c must have 2 dims, got " + std::to_string(c.dim()));
        check_size("c", c);
        const int64_t T = c.size(0);
        check_shape("c", c, {T, kLatent});
        check_shape("k_rope", r, {T, kRope});
        const kda_dtype code = code_of(cache);
        const ScalarType dt = cache.scalar_type();
        const int dev = device_of("cache", cache);
        const bool turned = a[4] != Py_None || a[5] != Py_None;
        if (turned && (a[4] == Py_None || a[5] == Py_None)) value_error("positions and inv_freq come together");
        const double factor = number(a[6]);
        const bool interleaved = truth(a[7]);
        int64_t cs, rs;
        const void *cp = lines("c", c, dev, dt, {T, kLatent}, cs), *rp = lines("k_rope", r, dev, dt, {T, kRope}, rs);
        void *kp = need("cache", cache, dev, dt, cache.sizes()), *sp = need("slot_map", slot, dev, kI64, {T}),
             *pp = turned ? need("positions", tensor("positions", a[4]), dev, kI32, {T}) : nullptr,
             *fp = turned ? need("inv_freq", tensor("inv_freq", a[5]), dev, kF32, {kRope / 2}) : nullptr;
        const Stream s = stream_of(a[8], dev);
        call("kda_latent_append", dev, [&] {
            return g_kda.latent_append(cp, rp, (const int64_t*)sp, (const int32_t*)pp, (const float*)fp, cs, rs, (int)T,
                                       (int)cache.size(1), (int)cache.size(0), interleaved, (float)factor, code, kp, s.handle);
        });
        Py_RETURN_NONE;
    });
}

PyObject* latent_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded("kda_latent_attention", n_args, 11, [&]() -> PyObject* {
        const Tensor &q = tensor("q", a[0]), &cache = tensor("cache", a[1]), &table = tensor("block_table", a[2]),
                     &cu = tensor("cu_seqlens", a[3]), &seq = tensor("seq_len", a[4]);
        check_latent_cache("kda_latent_attention", cache);
        if (q.dim() != 3 || table.dim() != 2)
            value_error("q must have 3 dims and block_table 2, got " + std::to_string(q.dim()) + " and " + std::to_string(table.dim()));
        check_size("q", q);
        check_size("block_table", table);
        const int64_t T = q.size(0), heads = q.size(1), n = table.size(0), blocks = table.size(1);
        check_shape("q", q, {T, heads, kLatent + kRope});
        check_shape("cu_seqlens", cu, {n + 1});
        check_shape("seq_len", seq, {n});
        const kda_dtype code = code_of(q);
        const ScalarType dt = q.scalar_type();
        const double scale = number(a[5]);
        const bool want_lse = a[7] != Py_None || truth(a[8]);
        const int dev = device_of("q", q);
        int64_t qs;
        const void* qp = rows("q", q, dev, dt, q.sizes(), qs);
        void *kp = need("cache", cache, dev, dt, cache.sizes()), *tp = need("block_table", table, dev, kI32, table.sizes()),
             *cup = need("cu_seqlens", cu, dev, kI32, {n + 1}), *sp = need("seq_len", seq, dev, kI32, {n});
        const Stream s = stream_of(a[10], dev);
        Tensor o = out("o", a[6], s, q, dt, {T, heads, kLatent}), lse;
        if (want_lse) lse = out("lse", a[7], s, q, kF32, {T, heads});
        size_t bytes = g_kda.latent_size((int)T, (int)heads, code);
        const Tensor ws = scratch(a[9], s, q, bytes);
        call("kda_latent_attention", dev, [&] {
            return g_kda.latent(qp, kp, (const int32_t*)tp, (const int32_t*)cup, (const int32_t*)sp, qs, (int)n, (int)T, (int)heads,
                                (int)cache.size(1), (int)blocks, (int)cache.size(0), (float)scale, code, o.data_ptr(),
                                want_lse ? (float*)lse.data_ptr() : nullptr, ws.data_ptr(), bytes, s.handle);
        });
        if (want_lse) return tuple({o, lse});
        return THPVariable_Wrap(o);
    });
}

PyObject* expanded_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded("kda_expanded_attention", n_args, 13, [&]() -> PyObject* {
        const Tensor &q = tensor("q", a[0]), &kn = tensor("k_nope", a[1]), &kr = tensor("k_rope", a[2]), &v = tensor("v", a[3]),
                     &cu = tensor("cu_seqlens", a[4]), &cuk = tensor("cu_seqlens_k", a[5]);
        if (q.dim() != 3 || v.dim() != 3 || cu.dim() != 1)
            value_error("q and v must have 3 dims and cu_seqlens 1, got " + std::to_string(q.dim()) + ", " + std::to_string(v.dim()) +
                        " and " + std::to_string(cu.dim()));
        check_size("q", q);
        check_size("v", v);
        check_size("cu_seqlens", cu);
        const int64_t T = q.size(0), heads = q.size(1), S = v.size(0), n = cu.size(0) - 1;
        if (n < 0) value_error("cu_seqlens must not be empty");
        check_shape("q", q, {T, heads, kNope + kRope});
        check_shape("k_nope", kn, {S, heads, kNope});
        check_shape("k_rope", kr, {S, kRope});
        check_shape("v", v, {S, heads, kValue});
        check_shape("cu_seqlens_k", cuk, {n + 1});
        const kda_dtype code = code_of(q);
        const ScalarType dt = q.scalar_type();
        const double scale = a[6] == Py_None ? 1.0 / std::sqrt((double)(kNope + kRope)) : number(a[6]);
        const bool causal = truth(a[7]), want_lse = a[9] != Py_None || truth(a[10]);
        const int dev = device_of("q", q);
        int64_t qs, knt, knh, krs, vt, vh;
        const void *qp = rows("q", q, dev, dt, q.sizes(), qs), *knp = strided("k_nope", kn, dev, dt, kn.sizes(), knt, knh),
                   *krp = lines("k_rope", kr, dev, dt, kr.sizes(), krs), *vp = strided("v", v, dev, dt, v.sizes(), vt, vh);
        void *cup = need("cu_seqlens", cu, dev, kI32, {n + 1}), *cukp = need("cu_seqlens_k", cuk, dev, kI32, {n + 1});
        const Stream s = stream_of(a[12], dev);
        Tensor o = out("o", a[8], s, q, dt, {T, heads, kValue}), lse;
        if (want_lse) lse = out("lse", a[9], s, q, kF32, {T, heads});
        size_t bytes = g_kda.expanded_size((int)T, (int)heads, code);
        const Tensor ws = scratch(a[11], s, q, bytes);
        call("kda_expanded_attention", dev, [&] {
            return g_kda.expanded(qp, knp, krp, vp, (const int32_t*)cup, (const int32_t*)cukp, qs, knt, knh, krs, vt, vh, (int)n,
                                  (int)T, (int)S, (int)heads, (float)scale, causal, code, o.data_ptr(),
                                  want_lse ? (float*)lse.data_ptr() : nullptr, ws.data_ptr(), bytes, s.handle);
        });
        if (want_lse) return tuple({o, lse});
        return THPVariable_Wrap(o);
    });
}

// set_entries(error class, C function addresses in the order of Entries): called once by _paged.py
constexpr int kEntries = 11;
PyObject* set_entries(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != kEntries + 1) {
        PyErr_SetString(PyExc_TypeError, "set_entries: wrong number of arguments");
        return nullptr;
    }
    void* p[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "set_entries: null entry");
            return nullptr;
        }
    }
    g_kda.tables = reinterpret_cast<decltype(g_kda.tables)>(p[0]);
    g_kda.append = reinterpret_cast<decltype(g_kda.append)>(p[1]);
    g_kda.attention_size = reinterpret_cast<decltype(g_kda.attention_size)>(p[2]);
    g_kda.attention = reinterpret_cast<decltype(g_kda.attention)>(p[3]);
    g_kda.verify = reinterpret_cast<decltype(g_kda.verify)>(p[4]);
    g_kda.rotary = reinterpret_cast<decltype(g_kda.rotary)>(p[5]);
    g_kda.latent_append = reinterpret_cast<decltype(g_kda.latent_append)>(p[6]);
    g_kda.latent_size = reinterpret_cast<decltype(g_kda.latent_size)>(p[7]);
    g_kda.latent = reinterpret_cast<decltype(g_kda.latent)>(p[8]);
    g_kda.expanded_size = reinterpret_cast<decltype(g_kda.expanded_size)>(p[9]);
    g_kda.expanded = reinterpret_cast<decltype(g_kda.expanded)>(p[10]);
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    Py_RETURN_NONE;
}

#define STEP_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {STEP_METHOD(set_entries),     STEP_METHOD(build_block_tables), STEP_METHOD(cache_append),
                           STEP_METHOD(paged_attention), STEP_METHOD(verify_draft),       STEP_METHOD(rotary),
                           STEP_METHOD(latent_append),   STEP_METHOD(latent_attention),   STEP_METHOD(expanded_attention),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_step_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step_binding(void) { return PyModule_Create(&g_module); }
