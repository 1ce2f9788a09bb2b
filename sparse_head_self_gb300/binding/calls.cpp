// The short way from Python into the calls whose work takes a few microseconds: a
// call of the usual form (tensors of torch itself on the current device and stream, results that
// the call makes) is checked and marshalled here, in about a third of what api.py's own steps
// take.  Each function returns None, before anything has happened, where a call is of another
// form or is to be refused: api.py then goes its way, with its messages.  A failed library call
// returns its status.
#include <Python.h>

#include <limits>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fibatt.h"

namespace {

// The library's functions, which the loader of the library hands over.
struct {
    decltype(&fibatt_window_fwd) window_fwd;
    decltype(&fibatt_window_bwd) window_bwd;
    decltype(&fibatt_window_bwd_workspace_bytes) window_ws;
    decltype(&fibatt_cache_store) cache_store;
    decltype(&fibatt_cache_load) cache_load;
    decltype(&fibatt_cache_fwd) cache_fwd;
} lib;

// A call's tensors: of one type, on the current device.
struct Call {
    bool ok = true;
    int index = -1;
    at::ScalarType type = at::kFloat;

    const at::Tensor *tensor(PyObject *o) {
        ok = ok && THPVariable_CheckExact(o);
        if (!ok) return nullptr;
        const at::Tensor &t = THPVariable_Unpack(o);
        ok = t.is_cuda() && t.layout() == at::kStrided;
        return &t;
    }
    // The first tensor, whose type and device the others have.
    const at::Tensor *first(PyObject *o) {
        const at::Tensor *t = tensor(o);
        if (!ok) return t;
        index = t->get_device();
        ok = index == c10::cuda::current_device();
        return t;
    }
    bool typed(const at::Tensor &t) {
        type = t.scalar_type();
        return ok = ok && (type == at::kFloat || type == at::kBFloat16);
    }
    fibatt_dtype dtype() const { return type == at::kFloat ? FIBATT_F32 : FIBATT_BF16; }
    // A tensor of heads [b, h, n, d].
    const at::Tensor *heads(PyObject *o, int64_t b, int64_t h, int64_t n, int64_t d, fibatt_heads *to) {
        const at::Tensor *t = tensor(o);
        if (ok) heads(*t, b, h, n, d, to);
        return t;
    }
    void heads(const at::Tensor &t, int64_t b, int64_t h, int64_t n, int64_t d, fibatt_heads *to) {
        ok = ok && t.scalar_type() == type && t.get_device() == index && t.dim() == 4;
        if (!ok) return;
        const auto s = t.sizes(), st = t.strides();
        ok = s[0] == b && s[1] == h && s[2] == n && s[3] == d && st[3] == 1;
        // a dim of one element has no stride that matters
        *to = fibatt_heads{t.data_ptr(), b > 1 ? st[0] : 0, h > 1 ? st[1] : 0, n > 1 ? st[2] : 0};
    }
    // One int32 a sequence, or None.
    const int32_t *numbers(PyObject *o, int64_t b) {
        if (o == Py_None) return nullptr;
        const at::Tensor *t = tensor(o);
        ok = ok && t->scalar_type() == at::kInt && t->get_device() == index && t->dim() == 1 && t->size(0) == b && t->is_contiguous();
        return ok ? static_cast<const int32_t *>(t->data_ptr()) : nullptr;
    }
    double number(PyObject *o) {
        ok = ok && PyFloat_CheckExact(o);
        return ok ? PyFloat_AS_DOUBLE(o) : 0.0;
    }
    // An int, or None for all.
    int whole(PyObject *o, bool none) {
        if (none && o == Py_None) return std::numeric_limits<int>::max();
        ok = ok && PyLong_CheckExact(o);
        if (!ok) return 0;
        int beyond = 0;
        const long v = PyLong_AsLongAndOverflow(o, &beyond);
        if (beyond > 0 || v > std::numeric_limits<int>::max()) return std::numeric_limits<int>::max();
        if (beyond < 0 || v < 0) ok = false;
        return (int)v;
    }
    int size(int64_t v) {
        ok = ok && v <= std::numeric_limits<int>::max();
        return (int)v;
    }
    cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
        return at::empty(shape, at::TensorOptions().dtype(t).device(at::kCUDA, (c10::DeviceIndex)index));
    }
};

PyObject *results(std::initializer_list<at::Tensor> ts) {
    PyObject *out = PyTuple_New((Py_ssize_t)ts.size());
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *o = THPVariable_Wrap(t);
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}
PyObject *refused(fibatt_status st) { return PyLong_FromLong(st); }

// The library's call without the interpreter's lock (a launch may wait for room in the stream).
template <typename F, typename... Args>
fibatt_status run(F f, Args... args) {
    PyThreadState *const state = PyEval_SaveThread();
    const fibatt_status st = f(args...);
    PyEval_RestoreThread(state);
    return st;
}

struct Window {
    Call c;
    fibatt_window d = {};
    fibatt_heads q, k, v;
    const at::Tensor *Q, *K, *V;
    // Q, K, V; scale, window, sinks, q_start, kv_len
    Window(PyObject *const *t, PyObject *const *how) {
        Q = c.first(t[0]), K = c.tensor(t[1]), V = c.tensor(t[2]);
        if (!c.ok || !c.typed(*Q) || Q->dim() != 4 || K->dim() != 4) {
            c.ok = false;
            return;
        }
        const auto sq = Q->sizes(), sk = K->sizes();
        d.B = c.size(sq[0]), d.Hq = c.size(sq[1]), d.Nq = c.size(sq[2]), d.D = c.size(sq[3]);
        d.Hkv = c.size(sk[1]), d.Nk = c.size(sk[2]);
        d.dtype = c.dtype();
        c.heads(*Q, sq[0], sq[1], sq[2], sq[3], &q);
        c.heads(*K, sq[0], sk[1], sk[2], sq[3], &k);
        c.heads(*V, sq[0], sk[1], sk[2], sq[3], &v);
        d.scale = (float)c.number(how[0]);
        d.window = c.whole(how[1], true);
        d.sinks = c.whole(how[2], false);
        d.q_start = c.numbers(how[3], sq[0]);
        d.kv_len = c.numbers(how[4], sq[0]);
    }
};

PyObject *window_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) Py_RETURN_NONE;
    Window w(a, a + 3);
    if (!w.c.ok) Py_RETURN_NONE;
    const at::Tensor O = at::empty_like(*w.Q), LSE = w.c.empty({w.d.B, w.d.Hq, w.d.Nq}, at::kFloat);
    fibatt_heads o;
    w.c.heads(O, w.d.B, w.d.Hq, w.d.Nq, w.d.D, &o);
    if (!w.c.ok) Py_RETURN_NONE;
    const fibatt_status st = run(lib.window_fwd, &w.d, &w.q, &w.k, &w.v, &o, static_cast<float *>(LSE.data_ptr()), w.c.stream());
    return st == FIBATT_OK ? results({O, LSE}) : refused(st);
    END_HANDLE_TH_ERRORS
}

// Q, K, V, O, LSE, dO, then as above
PyObject *window_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 11) Py_RETURN_NONE;
    Window w(a, a + 6);
    Call &c = w.c;
    if (!c.ok) Py_RETURN_NONE;
    fibatt_heads o, g, dq, dk, dv;
    c.heads(a[3], w.d.B, w.d.Hq, w.d.Nq, w.d.D, &o);
    c.heads(a[5], w.d.B, w.d.Hq, w.d.Nq, w.d.D, &g);
    const at::Tensor *LSE = c.tensor(a[4]);
    c.ok = c.ok && LSE->scalar_type() == at::kFloat && LSE->get_device() == c.index && LSE->is_contiguous() &&
           LSE->sizes() == w.Q->sizes().slice(0, 3);
    if (!c.ok) Py_RETURN_NONE;
    const at::Tensor dQ = at::empty_like(*w.Q), dK = at::empty_like(*w.K), dV = at::empty_like(*w.V);
    c.heads(dQ, w.d.B, w.d.Hq, w.d.Nq, w.d.D, &dq);
    c.heads(dK, w.d.B, w.d.Hkv, w.d.Nk, w.d.D, &dk);
    c.heads(dV, w.d.B, w.d.Hkv, w.d.Nk, w.d.D, &dv);
    if (!c.ok) Py_RETURN_NONE;
    const size_t need = lib.window_ws(&w.d);
    const at::Tensor ws = c.empty({(int64_t)need}, at::kByte);
    const fibatt_status st = run(lib.window_bwd, &w.d, &w.q, &w.k, &w.v, &o, static_cast<const float *>(LSE->data_ptr()), &g, &dq, &dk,
                                            &dv, ws.data_ptr(), need, c.stream());
    return st == FIBATT_OK ? results({dQ, dK, dV}) : refused(st);
    END_HANDLE_TH_ERRORS
}

// data, scales, table, start, count of a call of N tokens; the first tensor is known
bool cache(Call &c, fibatt_cache &d, PyObject *data, PyObject *scales, PyObject *table, PyObject *start, PyObject *count, int64_t B,
           int64_t N, int64_t D) {
    const at::Tensor *x = c.tensor(data), *s = c.tensor(scales), *t = c.tensor(table);
    if (!c.ok) return false;
    c.ok = x->scalar_type() == at::kByte && x->get_device() == c.index && x->dim() == 4 && x->size(2) == 2 &&
           x->size(3) == FIBATT_CACHE_PAGE * FIBATT_HEAD_DIM && x->is_contiguous() && s->scalar_type() == at::kFloat &&
           s->get_device() == c.index && s->is_contiguous() && s->sizes() == x->sizes().slice(0, 3) &&
           t->scalar_type() == at::kInt && t->get_device() == c.index && t->dim() == 2 && t->size(0) == B &&
           (t->size(1) == 1 || t->stride(1) == 1);
    if (!c.ok) return false;
    d.B = c.size(B), d.Hkv = c.size(x->size(1)), d.N = c.size(N), d.D = c.size(D);
    d.dtype = c.dtype();
    d.pages = c.size(x->size(0)), d.table_len = c.size(t->size(1));
    d.data = x->data_ptr();
    d.scales = static_cast<float *>(s->data_ptr());
    d.table = static_cast<const int32_t *>(t->data_ptr());
    d.table_stride_b = B > 1 ? t->stride(0) : 0;
    d.start = c.numbers(start, B);
    d.count = c.numbers(count, B);
    return c.ok;
}

// data, scales, table, K, V, start, count
PyObject *cache_store(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) Py_RETURN_NONE;
    Call c;
    fibatt_cache d = {};
    const at::Tensor *K = c.first(a[3]);
    if (!c.ok || !c.typed(*K) || K->dim() != 4) Py_RETURN_NONE;
    const auto s = K->sizes();
    fibatt_heads k, v;
    if (!cache(c, d, a[0], a[1], a[2], a[5], a[6], s[0], s[2], s[3])) Py_RETURN_NONE;
    c.heads(*K, s[0], d.Hkv, s[2], s[3], &k);
    c.heads(a[4], s[0], d.Hkv, s[2], s[3], &v);
    if (!c.ok) Py_RETURN_NONE;
    return refused(run(lib.cache_store, &d, &k, &v, c.stream()));
    END_HANDLE_TH_ERRORS
}

// data, scales, table, N, start, count, whether in 32 bits
PyObject *cache_load(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) Py_RETURN_NONE;
    Call c;
    fibatt_cache d = {};
    const at::Tensor *x = c.first(a[0]), *t = c.tensor(a[2]);
    const int N = c.whole(a[3], false);
    if (!c.ok || N < 1 || x->dim() != 4 || t->dim() != 2) Py_RETURN_NONE;
    c.type = a[6] == Py_True ? at::kFloat : at::kBFloat16;
    if (!cache(c, d, a[0], a[1], a[2], a[4], a[5], t->size(0), N, FIBATT_HEAD_DIM)) Py_RETURN_NONE;
    const at::Tensor K = c.empty({d.B, d.Hkv, N, FIBATT_HEAD_DIM}, c.type), V = at::empty_like(K);
    fibatt_heads k, v;
    c.heads(K, d.B, d.Hkv, N, FIBATT_HEAD_DIM, &k);
    c.heads(V, d.B, d.Hkv, N, FIBATT_HEAD_DIM, &v);
    if (!c.ok) Py_RETURN_NONE;
    const fibatt_status st = run(lib.cache_load, &d, &k, &v, c.stream());
    return st == FIBATT_OK ? results({K, V}) : refused(st);
    END_HANDLE_TH_ERRORS
}

// Q, data, scales, table, start, scale, window, sinks, count
PyObject *cache_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) Py_RETURN_NONE;
    Call c;
    fibatt_cache d = {};
    const at::Tensor *Q = c.first(a[0]);
    if (!c.ok || !c.typed(*Q) || Q->dim() != 4) Py_RETURN_NONE;
    const auto s = Q->sizes();
    fibatt_heads q, o;
    if (!cache(c, d, a[1], a[2], a[3], a[4], a[8], s[0], s[2], s[3])) Py_RETURN_NONE;
    c.heads(*Q, s[0], s[1], s[2], s[3], &q);
    const float scale = (float)c.number(a[5]);
    const int window = c.whole(a[6], true), sinks = c.whole(a[7], false), Hq = c.size(s[1]);
    if (!c.ok) Py_RETURN_NONE;
    const at::Tensor O = at::empty_like(*Q), LSE = c.empty({s[0], s[1], s[2]}, at::kFloat);
    c.heads(O, s[0], s[1], s[2], s[3], &o);
    if (!c.ok) Py_RETURN_NONE;
    const fibatt_status st =
        run(lib.cache_fwd, &d, Hq, scale, window, sinks, &q, &o, static_cast<float *>(LSE.data_ptr()), c.stream());
    return st == FIBATT_OK ? results({O, LSE}) : refused(st);
    END_HANDLE_TH_ERRORS
}

// The functions' addresses, in the order above.
PyObject *use(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "use() takes the addresses of six functions");
        return nullptr;
    }
    void *p[6];
    for (int i = 0; i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
            return nullptr;
        }
    }
    lib.window_fwd = reinterpret_cast<decltype(lib.window_fwd)>(p[0]);
    lib.window_bwd = reinterpret_cast<decltype(lib.window_bwd)>(p[1]);
    lib.window_ws = reinterpret_cast<decltype(lib.window_ws)>(p[2]);
    lib.cache_store = reinterpret_cast<decltype(lib.cache_store)>(p[3]);
    lib.cache_load = reinterpret_cast<decltype(lib.cache_load)>(p[4]);
    lib.cache_fwd = reinterpret_cast<decltype(lib.cache_fwd)>(p[5]);
    Py_RETURN_NONE;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    METHOD(use),
    METHOD(window_fwd),
    METHOD(window_bwd),
    METHOD(cache_store),
    METHOD(cache_load),
    METHOD(cache_fwd),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
