// kq_calls.cpp — the binding's fast path for the operators between a
// layer's products.  They are called once or more per layer and token and
// take a few microseconds on the GPU, while reading ten tensors' attributes
// and marshalling as many arguments from Python takes as long again.
//
// Each function takes the tensors as they are and calls the C ABI on the
// current stream, or returns None where anything is not plain (another
// device than the current one, another type or shape, a stride that the ABI
// does not take): the Python code then makes its own checks, and raises or
// calls.  Otherwise it returns the status.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kq.h"

namespace {

decltype(&kq_kv_plan) plan_fn = nullptr;
decltype(&kq_kv_append) append_fn = nullptr;
decltype(&kq_kv_attn) attn_fn = nullptr;
decltype(&kq_residual_norm) residual_fn = nullptr;

// The arguments of a call, read in order; `ok` falls when one is not plain.
struct Args {
    PyObject* const* a;
    int dev;
    bool ok = true;

    const at::Tensor* tensor(int i, at::ScalarType t) {
        if (!THPVariable_Check(a[i])) {
            ok = false;
            return nullptr;
        }
        const at::Tensor& x = THPVariable_Unpack(a[i]);
        if (!x.is_cuda() || x.get_device() != dev || x.scalar_type() != t || x.layout() != at::kStrided) {
            ok = false;
            return nullptr;
        }
        return &x;
    }
    bool none(int i) const { return a[i] == Py_None; }
    // a contiguous tensor of n elements (n < 0: any number)
    template <typename T>
    T* vec(int i, at::ScalarType t, int64_t n) {
        const at::Tensor* x = tensor(i, t);
        if (!x || (n >= 0 && x->numel() != n) || !x->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return static_cast<T*>(x->data_ptr());
    }
    template <typename T>
    T* opt(int i, at::ScalarType t, int64_t n) {
        return none(i) ? nullptr : vec<T>(i, t, n);
    }
    // a rows x cols tensor with contiguous rows
    template <typename T>
    T* mat(int i, at::ScalarType t, int64_t rows, int64_t cols, int64_t* ld) {
        const at::Tensor* x = tensor(i, t);
        if (!x || x->dim() != 2 || x->size(0) != rows || x->size(1) != cols || (cols > 1 && x->stride(1) != 1)) {
            ok = false;
            return nullptr;
        }
        *ld = rows > 1 ? x->stride(0) : cols;
        return static_cast<T*>(x->data_ptr());
    }
    int64_t integer(int i) {
        const long long v = PyLong_Check(a[i]) ? PyLong_AsLongLong(a[i]) : (ok = false, 0);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    int i32(int i) {
        const int64_t v = integer(i);
        if (v < INT32_MIN || v > INT32_MAX) ok = false;
        return static_cast<int>(v);
    }
    float real(int i) {
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return static_cast<float>(v);
    }
    kq_stream_t stream() const {
        return reinterpret_cast<kq_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
    }
};

constexpr at::ScalarType F32 = at::kFloat, I32 = at::kInt, I64 = at::kLong;

// Runs `body(args)`, which returns a status, or gives None.
template <typename F>
PyObject* call(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, int first_tensor, F body) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        if (THPVariable_Check(a[first_tensor])) {
            const at::Tensor& x = THPVariable_Unpack(a[first_tensor]);
            if (x.is_cuda() && x.get_device() == c10::cuda::current_device()) {
                Args g{a, static_cast<int>(x.get_device())};
                const int st = body(g);
                if (g.ok) return PyLong_FromLong(st);
            }
        }
    } catch (...) {  // (a tensor without plain storage, say)
    }
    Py_RETURN_NONE;
}

// (lens, add, table, free_pages, n_free, page_size, the plan's lens, q_start, slots, pos, n_left, status)
PyObject* py_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 12, 0, [](Args& g) {
        const at::Tensor *lens = g.tensor(0, I32), *table = g.tensor(2, I32), *stack = g.tensor(3, I32), *slots = g.tensor(8, I64);
        if (!g.ok || table->dim() != 2) return g.ok = false, 0;
        const int64_t R = lens->numel(), T = slots->numel(), width = table->size(1), cap = stack->numel();
        if (R > INT32_MAX - 1 || width > INT32_MAX || cap > INT32_MAX) return g.ok = false, 0;
        int64_t ld = 0;
        int32_t* tab = g.mat<int32_t>(2, I32, R, width, &ld);
        const int32_t *len = g.vec<int32_t>(0, I32, R), *add = g.vec<int32_t>(1, I32, R), *free = g.vec<int32_t>(3, I32, cap),
                      *n_free = g.vec<int32_t>(4, I32, 1);
        const int page = g.i32(5);
        int32_t *nl = g.vec<int32_t>(6, I32, R), *qs = g.vec<int32_t>(7, I32, R + 1);
        int64_t* sl = g.vec<int64_t>(8, I64, T);
        int32_t *pos = g.vec<int32_t>(9, I32, T), *left = g.vec<int32_t>(10, I32, 1), *st = g.opt<int32_t>(11, I32, 1);
        if (!g.ok) return 0;
        return plan_fn(static_cast<int>(R), len, add, page, tab, ld, static_cast<int>(width), free, static_cast<int>(cap), n_free,
                       T, nl, qs, sl, pos, left, st, g.stream());
    });
}

// (qkv, n_q, cache, slots, pos, inv_freq, adjacent, q_gamma, k_gamma, eps, q_out, status, the cache's device)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 13, 0, [](Args& g) {
        const at::Tensor* x = g.tensor(0, F32);
        if (g.i32(12) != g.dev) return g.ok = false, 0;
        const int n_q = g.i32(1);
        const auto* c = reinterpret_cast<const kq_kv_cache*>(g.integer(2));
        if (!g.ok || x->dim() != 2 || n_q < 1 || n_q > 65535 || c->n_kv < 1 || c->n_kv > 65535) return g.ok = false, 0;
        const int64_t T = x->size(0), D = c->head_dim;
        int64_t ld = 0, ldq = 0;
        const float* qkv = g.mat<float>(0, F32, T, (n_q + 2 * static_cast<int64_t>(c->n_kv)) * D, &ld);
        const int64_t* slots = g.vec<int64_t>(3, I64, T);
        const int32_t* pos = g.vec<int32_t>(4, I32, T);
        kq_rotary rot{};
        if (!g.none(5)) {
            rot.inv_freq = g.vec<float>(5, F32, -1);
            if (!g.ok) return 0;
            const int64_t half = THPVariable_Unpack(g.a[5]).numel();
            if (half > 65535) return g.ok = false, 0;
            rot.rot_dim = static_cast<int>(2 * half);
        }
        rot.adjacent = g.i32(6);
        rot.q_gamma = g.opt<float>(7, F32, D);
        rot.k_gamma = g.opt<float>(8, F32, D);
        rot.eps = g.real(9);
        float* q = g.mat<float>(10, F32, T, n_q * D, &ldq);
        int32_t* st = g.opt<int32_t>(11, I32, 1);
        if (!g.ok) return 0;
        return append_fn(T, qkv, ld, n_q, c, slots, pos, &rot, q, ldq, st, g.stream());
    });
}

// (q, cache, lens, table, q_start, max_q, scale, window, out, workspace, status, the cache's device)
PyObject* py_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 12, 0, [](Args& g) {
        if (g.i32(11) != g.dev) return g.ok = false, 0;
        const at::Tensor *x = g.tensor(0, F32), *lens = g.tensor(2, I32), *table = g.tensor(3, I32);
        const auto* c = reinterpret_cast<const kq_kv_cache*>(g.integer(1));
        if (!g.ok || x->dim() != 2 || table->dim() != 2 || c->head_dim < 1) return g.ok = false, 0;
        const int64_t T = x->size(0), cols = x->size(1), n_q = cols / c->head_dim, R = lens->numel(), width = table->size(1);
        if (n_q * c->head_dim != cols || n_q > INT32_MAX || R > INT32_MAX - 1 || width > INT32_MAX) return g.ok = false, 0;
        int64_t ldq = 0, ldo = 0, ldt = 0;
        const float* q = g.mat<float>(0, F32, T, cols, &ldq);
        const int32_t *len = g.vec<int32_t>(2, I32, R), *tab = g.mat<int32_t>(3, I32, R, width, &ldt),
                      *start = g.opt<int32_t>(4, I32, R + 1);
        const int max_q = g.i32(5);
        const float scale = g.real(6);
        const int window = g.i32(7);
        float* out = g.mat<float>(8, F32, T, cols, &ldo);
        if (!THPVariable_Check(g.a[9])) return g.ok = false, 0;
        const at::Tensor& ws = THPVariable_Unpack(g.a[9]);
        if (!ws.is_cuda() || ws.get_device() != g.dev || !ws.is_contiguous()) return g.ok = false, 0;
        int32_t* st = g.opt<int32_t>(10, I32, 1);
        if (!g.ok) return 0;
        return attn_fn(static_cast<int>(R), T, max_q, static_cast<int>(n_q), q, ldq, c, len, start, tab, ldt,
                       static_cast<int>(width), scale, window, out, ldo, ws.data_ptr(), static_cast<size_t>(ws.nbytes()), st,
                       g.stream());
    });
}

// (out, res, y, weights, post_gamma, gate, scale, pre_gamma, eps, h)
PyObject* py_residual(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 10, 0, [](Args& g) {
        const at::Tensor* o = g.tensor(0, F32);
        if (!g.ok || o->dim() != 2 || (g.none(1) && g.none(2))) return g.ok = false, 0;
        const int64_t T = o->size(0), N = o->size(1);
        kq_residual r{};
        r.out = g.mat<float>(0, F32, T, N, &r.ldout);
        if (!g.none(1)) r.res = g.mat<float>(1, F32, T, N, &r.ldres);
        if (!g.none(2)) {
            const at::Tensor* y = g.tensor(2, F32);
            if (!g.ok) return 0;
            if (y->dim() == 2) {
                r.n_terms = 1;
                r.y = g.mat<float>(2, F32, T, N, &r.ldy);
                r.ld_term = N;
            } else {
                if (y->dim() != 3 || y->size(0) != T || y->size(2) != N || (N > 1 && y->stride(2) != 1) || y->size(1) > 65535)
                    return g.ok = false, 0;
                r.n_terms = static_cast<int>(y->size(1));
                r.y = static_cast<const float*>(y->data_ptr());
                r.ldy = T > 1 ? y->stride(0) : r.n_terms * N;
                r.ld_term = r.n_terms > 1 ? y->stride(1) : N;
            }
            if (!g.none(3)) r.weights = g.mat<float>(3, F32, T, r.n_terms, &r.ldw);
        } else if (!g.none(3)) {
            return g.ok = false, 0;
        }
        r.post_gamma = g.opt<float>(4, F32, N);
        if (!g.none(5)) {
            const at::Tensor* gate = g.tensor(5, F32);
            if (!g.ok) return 0;
            if (gate->dim() == 1) r.gate = g.vec<float>(5, F32, N);
            else r.gate = g.mat<float>(5, F32, T, N, &r.ldg);
        }
        r.scale = g.real(6);
        r.pre_gamma = g.opt<float>(7, F32, N);
        r.eps = g.real(8);
        if (!g.none(9)) r.h = g.mat<float>(9, F32, T, N, &r.ldh);
        if (!g.ok) return 0;
        return residual_fn(&r, T, N, g.stream());
    });
}

// The C ABI's addresses in the library that the binding has loaded.
PyObject* py_use(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[4];
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "use() takes 4 addresses");
        return nullptr;
    }
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    plan_fn = reinterpret_cast<decltype(plan_fn)>(p[0]);
    append_fn = reinterpret_cast<decltype(append_fn)>(p[1]);
    attn_fn = reinterpret_cast<decltype(attn_fn)>(p[2]);
    residual_fn = reinterpret_cast<decltype(residual_fn)>(p[3]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"use", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_use)), METH_FASTCALL, nullptr},
    {"kv_plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_plan)), METH_FASTCALL, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_append)), METH_FASTCALL, nullptr},
    {"kv_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_attn)), METH_FASTCALL, nullptr},
    {"residual_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_residual)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
    PyObject* m = PyModule_Create(&module);
    // what this file was built against; the binding takes it for nothing else
    if (m && PyModule_AddStringConstant(m, "key", KQ_CALLS_KEY) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
