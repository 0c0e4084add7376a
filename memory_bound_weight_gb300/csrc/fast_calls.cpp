// fast_calls.cpp -- the binding's checks and marshalling of the calls that a
// decode step makes many times, in C++: kv4_append, kv4_gather, kv4_attention,
// kv4_attention_shared, token_logprobs, the 8-bit quantizers and products. Each function checks what the Python function of its name
// checks, allocates the outputs, makes the library's call on the current stream
// and returns the outputs, or the library's status where that is not 0. What it
// does not take as it is (a wrong argument, a tensor's subclass, a missing
// allocation) it answers with None and without any effect: the Python function
// then says what is wrong, or does the call. (Host time of attention of one request
// 15.6 us in Python and 9.8 here, of an append and a gather 27 and 18, of log
// probabilities with their five outputs 20 and 11.)
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mbw.h"

namespace {

decltype(&mbw_kv4_append) append_fn;
decltype(&mbw_kv4_gather) gather_fn;
decltype(&mbw_kv4_attention) attention_fn;
decltype(&mbw_kv4_attention_shared) shared_fn;
decltype(&mbw_token_logprobs) logprobs_fn;
decltype(&mbw_quantize_fp8_g128) rows_fn;
decltype(&mbw_quantize_fp8_b128) blocks_fn;
decltype(&mbw_dequant_fp8_g128) row_values_fn, block_values_fn;
decltype(&gemm_fp8_b128) product_fn;

struct Unusual {};  // left to the Python function

int device_now() { return c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index(); }

const at::Tensor* tensor(PyObject* o, int dev, at::ScalarType type) {
    if (!THPVariable_CheckExact(o)) throw Unusual();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type) throw Unusual();
    return &t;
}
const at::Tensor* plain(PyObject* o, int dev, at::ScalarType type, int dims) {
    const at::Tensor* t = tensor(o, dev, type);
    if (t->dim() != dims || !t->is_contiguous()) throw Unusual();
    return t;
}
const at::Tensor* vector(PyObject* o, int dev, at::ScalarType type, int64_t n) {
    const at::Tensor* t = plain(o, dev, type, 1);
    if (t->size(0) != n) throw Unusual();
    return t;
}
struct Rows {  // bf16 (n, heads, dim), possibly rows of a wider matrix
    const at::Tensor* t;
    int64_t n, heads, stride;
};
Rows rows(PyObject* o, int dev, int64_t heads, int64_t dim) {
    const at::Tensor* t = tensor(o, dev, at::kBFloat16);
    if (t->dim() != 3) throw Unusual();
    const int64_t n = t->size(0), h = t->size(1);
    if (t->size(2) != dim || (heads >= 0 && h != heads) || t->stride(2) != 1 || (t->stride(1) != dim && h != 1)) throw Unusual();
    return {t, n, h, n > 1 ? t->stride(0) : h * dim};
}
void* workspace(PyObject* o, int dev, size_t& bytes) {
    bytes = 0;
    if (o == Py_None) return nullptr;
    if (!THPVariable_CheckExact(o)) throw Unusual();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous()) throw Unusual();
    bytes = t.nbytes();
    return t.data_ptr();
}
// The cache's struct, if its tensor still lies where it lay when that was made.
const mbw_kv4_cache* cache_of(PyObject* addr, PyObject* pages, int dev) {
    const at::Tensor* t = plain(pages, dev, at::kByte, 2);
    const mbw_kv4_cache* c = static_cast<const mbw_kv4_cache*>(PyLong_AsVoidPtr(addr));
    if (!c || t->data_ptr() != c->pages || t->size(0) != c->num_pages) throw Unusual();
    return c;
}
int64_t whole(PyObject* o) {
    if (!PyLong_CheckExact(o)) throw Unusual();
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Unusual();
    return v;
}
double number(PyObject* o) {
    if (!PyFloat_CheckExact(o)) throw Unusual();
    return PyFloat_AS_DOUBLE(o);
}
mbw_stream_t stream(int dev) { return (mbw_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
at::Tensor empty(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type) { return at::empty(shape, like.options().dtype(type)); }

template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (...) {  // a C++ exception does not pass into the interpreter
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// (address of the cache's struct, pages, k, v, slots, q, positions, cos_sin, interleaved, q_out)
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 10) throw Unusual();
        const int dev = device_now();
        const mbw_kv4_cache* c = cache_of(a[0], a[1], dev);
        const int64_t d = c->head_dim;
        const Rows k = rows(a[2], dev, c->kv_heads, d), v = rows(a[3], dev, c->kv_heads, d);
        if (v.n != k.n) throw Unusual();
        const at::Tensor* slots = vector(a[4], dev, at::kLong, k.n);
        if ((a[6] == Py_None) != (a[7] == Py_None) || (a[5] == Py_None && a[9] != Py_None)) throw Unusual();
        mbw_rope rope{};
        if (a[6] != Py_None) {
            const at::Tensor *pos = vector(a[6], dev, at::kInt, k.n), *cs = plain(a[7], dev, at::kFloat, 2);
            const int il = PyObject_IsTrue(a[8]);
            if (il < 0 || cs->size(1) > INT32_MAX) throw Unusual();
            rope = {cs->data_ptr<float>(), cs->size(0), (int32_t)cs->size(1), il, pos->data_ptr<int32_t>()};
        }
        Rows q{}, to{};
        at::Tensor made;
        if (a[5] != Py_None) {
            q = rows(a[5], dev, -1, d);
            if (q.n != k.n) throw Unusual();
            if (a[9] == Py_None) {
                made = empty({q.n, q.heads, d}, *q.t, at::kBFloat16);
                to = {&made, q.n, q.heads, q.heads * d};
            } else {
                to = rows(a[9], dev, q.heads, d);
                if (to.n != q.n) throw Unusual();
            }
        }
        const mbw_status st = append_fn(c, k.t->data_ptr(), k.stride, v.t->data_ptr(), v.stride, slots->data_ptr<int64_t>(),
                                        q.t ? q.t->data_ptr() : nullptr, q.stride, q.t ? to.t->data_ptr() : nullptr, to.stride,
                                        q.heads, a[6] != Py_None ? &rope : nullptr, k.n, stream(dev));
        if (st) return PyLong_FromLong(st);
        PyObject* out = made.defined() ? THPVariable_Wrap(made) : (Py_INCREF(a[9]), a[9]);
        if (!out) return nullptr;
        PyObject* r = PyTuple_Pack(1, out);  // None is an answer here
        Py_DECREF(out);
        return r;
    });
}

// (address, pages, slots)
PyObject* kv4_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 3) throw Unusual();
        const int dev = device_now();
        const mbw_kv4_cache* c = cache_of(a[0], a[1], dev);
        const at::Tensor* slots = plain(a[2], dev, at::kLong, 1);
        const int64_t T = slots->size(0);
        const at::Tensor k = empty({T, c->kv_heads, c->head_dim}, *slots, at::kBFloat16), v = at::empty_like(k);
        const mbw_status st = gather_fn(c, slots->data_ptr<int64_t>(), k.data_ptr(), v.data_ptr(), T, stream(dev));
        if (st) return PyLong_FromLong(st);
        return Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v));
    });
}

// (address, pages, q, block_table, ctx_lens, q_starts, scale, window, return_lse, workspace[, shared_len])
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 10 && n != 11) throw Unusual();
        const int dev = device_now();
        const mbw_kv4_cache* c = cache_of(a[0], a[1], dev);
        const Rows q = rows(a[2], dev, -1, c->head_dim);
        const at::Tensor* table = plain(a[3], dev, at::kInt, 2);
        const int64_t B = table->size(0), width = table->size(1);
        const at::Tensor* ctx = vector(a[4], dev, at::kInt, B);
        const at::Tensor* starts = a[5] == Py_None ? nullptr : vector(a[5], dev, at::kInt, B + 1);
        const double scale = number(a[6]);
        const int64_t window = whole(a[7]);
        const int want_lse = PyObject_IsTrue(a[8]);
        if (want_lse < 0) throw Unusual();
        size_t bytes;
        void* ws = workspace(a[9], dev, bytes);
        const at::Tensor out = empty({q.n, q.heads, c->head_dim}, *q.t, at::kBFloat16);
        at::Tensor lse;
        if (want_lse) lse = empty({q.n, q.heads}, *q.t, at::kFloat);
        float* lse_at = want_lse ? lse.data_ptr<float>() : nullptr;
        const int32_t* starts_at = starts ? starts->data_ptr<int32_t>() : nullptr;
        const mbw_status st = n == 11 ? shared_fn(c, q.t->data_ptr(), q.stride, out.data_ptr(), q.heads * c->head_dim, lse_at, table->data_ptr<int32_t>(),
                                                  width, width, ctx->data_ptr<int32_t>(), starts_at, B, q.n, q.heads, (float)scale, window,
                                                  whole(a[10]), ws, bytes, stream(dev))
                                      : attention_fn(c, q.t->data_ptr(), q.stride, out.data_ptr(), q.heads * c->head_dim, lse_at,
                                                     table->data_ptr<int32_t>(), width, width, ctx->data_ptr<int32_t>(), starts_at, B, q.n, q.heads,
                                                     (float)scale, window, ws, bytes, stream(dev));
        if (st) return PyLong_FromLong(st);
        PyObject* o = THPVariable_Wrap(out);
        return want_lse ? Py_BuildValue("(NN)", o, THPVariable_Wrap(lse)) : o;
    });
}

// (logits, targets, top_k, scale, workspace)
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 5) throw Unusual();
        const int dev = device_now();
        if (!THPVariable_CheckExact(a[0])) throw Unusual();
        const bool wide = THPVariable_Unpack(a[0]).scalar_type() == at::kFloat;
        const at::Tensor* x = tensor(a[0], dev, wide ? at::kFloat : at::kBFloat16);
        if (x->dim() != 2) throw Unusual();
        const int64_t M = x->size(0), V = x->size(1), K = whole(a[2]);
        if ((x->stride(1) != 1 && V > 1) || K < 0 || K > 32) throw Unusual();
        const at::Tensor* targets = a[1] == Py_None ? nullptr : vector(a[1], dev, at::kInt, M);
        const double scale = number(a[3]);
        size_t bytes;
        void* ws = workspace(a[4], dev, bytes);
        at::Tensor lp, rank;
        if (targets) lp = empty({M}, *x, at::kFloat), rank = empty({M}, *x, at::kInt);
        const at::Tensor entropy = empty({M}, *x, at::kFloat), ids = empty({M, K}, *x, at::kInt), top = empty({M, K}, *x, at::kFloat);
        const mbw_status st = logprobs_fn(x->data_ptr(), wide, M > 1 ? x->stride(0) : V, targets ? targets->data_ptr<int32_t>() : nullptr,
                                          M, V, (float)scale, (int32_t)K, targets ? lp.data_ptr<float>() : nullptr,
                                          targets ? rank.data_ptr<int32_t>() : nullptr, entropy.data_ptr<float>(),
                                          ids.data_ptr<int32_t>(), top.data_ptr<float>(), ws, bytes, stream(dev));
        if (st) return PyLong_FromLong(st);
        auto wrap = [](const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : (Py_INCREF(Py_None), Py_None); };
        return Py_BuildValue("(NNNNN)", wrap(lp), wrap(rank), wrap(entropy), wrap(ids), wrap(top));
    });
}

// A matrix of e4m3 codes, whose width is a positive multiple of 128.
const at::Tensor* codes(PyObject* o, int dev) {
    const at::Tensor* t = plain(o, dev, at::kFloat8_e4m3fn, 2);
    if (t->size(1) % 128 || t->size(1) == 0) throw Unusual();
    return t;
}
const at::Tensor* matrix(PyObject* o, int dev, at::ScalarType type, int64_t rows, int64_t columns) {
    const at::Tensor* t = plain(o, dev, type, 2);
    if (t->size(0) != rows || t->size(1) != columns) throw Unusual();
    return t;
}

// (X, norm_weight, norm_eps)
PyObject* quantize_fp8_g128(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 3) throw Unusual();
        const int dev = device_now();
        const at::Tensor* x = tensor(a[0], dev, at::kBFloat16);
        if (x->dim() != 2 || x->stride(1) != 1) throw Unusual();
        const int64_t M = x->size(0), K = x->size(1);
        if (K % 128 || K == 0) throw Unusual();
        const at::Tensor* w = a[1] == Py_None ? nullptr : vector(a[1], dev, at::kBFloat16, K);
        const double eps = number(a[2]);
        const at::Tensor q = empty({M, K}, *x, at::kFloat8_e4m3fn), s = empty({M, K / 128}, *x, at::kFloat);
        const mbw_status st = rows_fn(x->data_ptr(), M > 1 ? x->stride(0) : K, static_cast<uint8_t*>(q.data_ptr()), s.data_ptr<float>(), M, K,
                                      w ? w->data_ptr() : nullptr, eps, stream(dev));
        if (st) return PyLong_FromLong(st);
        return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(s));
    });
}

// (W)
PyObject* quantize_fp8_b128(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 1) throw Unusual();
        const int dev = device_now();
        const at::Tensor* w = plain(a[0], dev, at::kBFloat16, 2);
        const int64_t N = w->size(0), K = w->size(1);
        if (K % 128 || K == 0) throw Unusual();
        const at::Tensor q = empty({N, K}, *w, at::kFloat8_e4m3fn), s = empty({(N + 127) / 128, K / 128}, *w, at::kFloat);
        const mbw_status st = blocks_fn(w->data_ptr(), static_cast<uint8_t*>(q.data_ptr()), s.data_ptr<float>(), N, K, stream(dev));
        if (st) return PyLong_FromLong(st);
        return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(s));
    });
}

// (codes, scales, rows of a scale: 1 or 128)
PyObject* dequant_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 3) throw Unusual();
        const int dev = device_now();
        const at::Tensor* q = codes(a[0], dev);
        const int64_t M = q->size(0), K = q->size(1), rows = whole(a[2]);
        const at::Tensor* s = matrix(a[1], dev, at::kFloat, (M + rows - 1) / rows, K / 128);
        const at::Tensor out = empty({M, K}, *q, at::kFloat);
        const mbw_status st = (rows == 1 ? row_values_fn : block_values_fn)(static_cast<const uint8_t*>(q->data_ptr()), s->data_ptr<float>(),
                                                                             out.data_ptr<float>(), M, K, stream(dev));
        return st ? PyLong_FromLong(st) : THPVariable_Wrap(out);
    });
}

// (Xq, x_scales, Wq, w_scales, residual, up_weights, up_scales, workspace)
PyObject* gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 8) throw Unusual();
        const int dev = device_now();
        const at::Tensor *x = codes(a[0], dev), *w = codes(a[2], dev);
        const int64_t M = x->size(0), K = x->size(1), N = w->size(0), blocks = (N + 127) / 128;
        if (w->size(1) != K) throw Unusual();
        const at::Tensor *xs = matrix(a[1], dev, at::kFloat, M, K / 128), *ws = matrix(a[3], dev, at::kFloat, blocks, K / 128);
        mbw_fusion f{};
        if (a[4] != Py_None) f.residual = matrix(a[4], dev, at::kBFloat16, M, N)->data_ptr();
        if ((a[5] == Py_None) != (a[6] == Py_None)) throw Unusual();
        if (a[5] != Py_None) {
            const at::Tensor* u = codes(a[5], dev);
            if (u->size(0) != N || u->size(1) != K) throw Unusual();
            f.up_weights = u->data_ptr();
            f.up_scales = matrix(a[6], dev, at::kFloat, blocks, K / 128)->data_ptr();
        }
        size_t bytes;
        void* space = workspace(a[7], dev, bytes);
        const at::Tensor y = empty({M, N}, *x, at::kBFloat16);
        const mbw_status st = product_fn(static_cast<const uint8_t*>(x->data_ptr()), xs->data_ptr<float>(), static_cast<const uint8_t*>(w->data_ptr()),
                                         ws->data_ptr<float>(), y.data_ptr(), M, N, K, &f, space, bytes, stream(dev));
        return st ? PyLong_FromLong(st) : THPVariable_Wrap(y);
    });
}

// The library's functions, by address.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 10) {
        PyErr_SetString(PyExc_TypeError, "ten addresses");
        return nullptr;
    }
    shared_fn = reinterpret_cast<decltype(shared_fn)>(PyLong_AsVoidPtr(a[4]));
    rows_fn = reinterpret_cast<decltype(rows_fn)>(PyLong_AsVoidPtr(a[5]));
    blocks_fn = reinterpret_cast<decltype(blocks_fn)>(PyLong_AsVoidPtr(a[6]));
    row_values_fn = reinterpret_cast<decltype(row_values_fn)>(PyLong_AsVoidPtr(a[7]));
    block_values_fn = reinterpret_cast<decltype(block_values_fn)>(PyLong_AsVoidPtr(a[8]));
    product_fn = reinterpret_cast<decltype(product_fn)>(PyLong_AsVoidPtr(a[9]));
    append_fn = reinterpret_cast<decltype(append_fn)>(PyLong_AsVoidPtr(a[0]));
    gather_fn = reinterpret_cast<decltype(gather_fn)>(PyLong_AsVoidPtr(a[1]));
    attention_fn = reinterpret_cast<decltype(attention_fn)>(PyLong_AsVoidPtr(a[2]));
    logprobs_fn = reinterpret_cast<decltype(logprobs_fn)>(PyLong_AsVoidPtr(a[3]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", (PyCFunction)(void*)init, METH_FASTCALL, nullptr},
    {"kv4_append", (PyCFunction)(void*)kv4_append, METH_FASTCALL, nullptr},
    {"kv4_gather", (PyCFunction)(void*)kv4_gather, METH_FASTCALL, nullptr},
    {"kv4_attention", (PyCFunction)(void*)kv4_attention, METH_FASTCALL, nullptr},
    {"token_logprobs", (PyCFunction)(void*)token_logprobs, METH_FASTCALL, nullptr},
    {"quantize_fp8_g128", (PyCFunction)(void*)quantize_fp8_g128, METH_FASTCALL, nullptr},
    {"quantize_fp8_b128", (PyCFunction)(void*)quantize_fp8_b128, METH_FASTCALL, nullptr},
    {"dequant_fp8", (PyCFunction)(void*)dequant_fp8, METH_FASTCALL, nullptr},
    {"gemm_fp8", (PyCFunction)(void*)gemm_fp8, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `built_for`, by which the binding knows whether these calls fit the PyTorch that runs.
PyMODINIT_FUNC PyInit__fast(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", MBW_BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
