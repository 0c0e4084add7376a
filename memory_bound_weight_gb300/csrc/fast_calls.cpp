// fast_calls.cpp -- the binding's checks and marshalling of the calls that a
// decode step makes many times, in C++: kv4_append, kv4_gather, kv4_attention
// and token_logprobs. Each function checks what the Python function of its name
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
decltype(&mbw_token_logprobs) logprobs_fn;

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

// (address, pages, q, block_table, ctx_lens, q_starts, scale, window, return_lse, workspace)
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 10) throw Unusual();
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
        const mbw_status st = attention_fn(c, q.t->data_ptr(), q.stride, out.data_ptr(), q.heads * c->head_dim,
                                           want_lse ? lse.data_ptr<float>() : nullptr, table->data_ptr<int32_t>(), width, width,
                                           ctx->data_ptr<int32_t>(), starts ? starts->data_ptr<int32_t>() : nullptr, B, q.n,
                                           q.heads, (float)scale, window, ws, bytes, stream(dev));
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

// The library's functions, by address.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "four addresses");
        return nullptr;
    }
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
