// calls.cpp -- the short way into the library for calls of a few microseconds
// of GPU work (the row kernels and the int8 product): a CPython module that
// checks the tensors, allocates the outputs and calls the C entry point.
//
// Each function takes the Python function's arguments in order and returns its
// result; or None where anything does not fit (a type, a shape, a device that
// is not the current one, a tensor subclass, a vector not on 16 bytes), which ops.py then does or refuses
// the long way, with its messages; or, as an integer, the status that the
// entry point returned.  By ctypes and Python's tensor attributes fwd_q8 took
// 10.1 us, of which the entry point with its launch is 3.0.
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include "../../include/slope.h"

// What this was built for, as build.py looks for it.
extern "C" __attribute__((used, visibility("default"))) const char slope_calls_key[] = "slope calls for " SLOPE_CALLS_KEY;

namespace {

// The entry points of the library that ops.py loaded (release or debug build).
struct Entry {
    decltype(&slope_rmsnorm) rmsnorm;
    decltype(&slope_rmsnorm_bwd) rmsnorm_bwd;
    decltype(&slope_rmsnorm_bwd_ws) rmsnorm_bwd_ws;
    decltype(&slope_quant_rows) quant_rows;
    decltype(&slope_fwd_q8) fwd_q8;
} lib = {};

// The tensor of a Python object if it is a contiguous CUDA one of `type` and `dims` dimensions, else null.
const at::Tensor *plain(PyObject *o, at::ScalarType type, int64_t dims) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.defined() || t.scalar_type() != type || !t.is_cuda() || t.layout() != at::kStrided || t.dim() != dims || !t.is_contiguous())
        return nullptr;
    return &t;
}

// One call: the arguments' device, and whether everything has fitted so far.
struct Call {
    int dev = -1;
    bool fits = true;

    explicit Call(const at::Tensor *first) {
        fits = lib.rmsnorm && first && first->get_device() == c10::cuda::current_device();  // bound, and here
        if (fits) dev = first->get_device();
    }
    template <typename T>
    T *in(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor *t = fits ? plain(o, type, (int64_t)shape.size()) : nullptr;
        if (!t || t->get_device() != dev || t->sizes() != at::IntArrayRef(shape)) {
            fits = false;
            return nullptr;
        }
        T *p = static_cast<T *>(t->data_ptr());
        // an fp32 vector may be a slice, which ops.py copies
        if (type == at::kFloat && (reinterpret_cast<uintptr_t>(p) & 15u)) fits = false;
        return p;
    }
    // whether an output that the caller gave fits (None: one will be allocated)
    void given(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> shape) {
        if (o != Py_None) in<void>(o, type, shape);
    }
    // the output, given or new, as a new reference in `result`
    template <typename T>
    T *out(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> shape, PyObject *&result) {
        if (o != Py_None) {
            Py_INCREF(o);
            result = o;
            return static_cast<T *>(THPVariable_Unpack(o).data_ptr());
        }
        at::Tensor t = fresh(type, shape);
        T *p = static_cast<T *>(t.data_ptr());
        result = THPVariable_Wrap(std::move(t));
        return p;
    }
    at::Tensor fresh(at::ScalarType type, std::initializer_list<int64_t> shape) const {
        return at::detail::empty_cuda(at::IntArrayRef(shape), type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

// References that are dropped unless the call succeeds.
struct Results {
    static constexpr int MOST = 5;
    PyObject *o[MOST] = {};
    int n;
    explicit Results(int count) : n(count) {}
    ~Results() {
        for (PyObject *p : o) Py_XDECREF(p);
    }
    PyObject *take(int rc) {  // the status, the single result, or the tuple of them (None where there is none)
        if (rc != 0) return PyLong_FromLong(rc);
        if (n == 1) {
            PyObject *r = o[0];
            o[0] = nullptr;
            return r;
        }
        PyObject *t = PyTuple_New(n);
        if (!t) return nullptr;
        for (int i = 0; i < n; ++i) {
            if (!o[i]) {
                Py_INCREF(Py_None);
                o[i] = Py_None;
            }
            PyTuple_SET_ITEM(t, i, o[i]);
            o[i] = nullptr;
        }
        return t;
    }
};

// The call itself, without the interpreter's lock: a full launch queue may make it wait.
template <typename F>
int unlocked(F &&f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return rc;
}

// Integers and floats as Python's own numbers only.
bool as_int(PyObject *o, int64_t &v) {
    if (!PyLong_Check(o)) return false;
    int over = 0;
    v = PyLong_AsLongLongAndOverflow(o, &over);
    return over == 0;
}
bool as_float(PyObject *o, float &v) {
    if (!PyFloat_Check(o)) return false;
    v = (float)PyFloat_AS_DOUBLE(o);
    return true;
}

bool flag(PyObject *o, bool &fits) {  // True or False themselves
    if (o != Py_True && o != Py_False) fits = false;
    return o == Py_True;
}

// rmsnorm(X, w, eps, res, with_y, with_q8, with_rstd, H, Y, Q, qscale, rstd) -> (Q, qscale, Y, H, rstd)
PyObject *rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    float eps;
    const at::Tensor *x = n == 12 ? plain(a[0], at::kBFloat16, 2) : nullptr;
    Call c(x);
    if (!c.fits || !as_float(a[2], eps)) Py_RETURN_NONE;
    const int64_t T = x->size(0), D = x->size(1);
    const bool res = a[3] != Py_None, y = flag(a[4], c.fits), q8 = flag(a[5], c.fits);
    const bool r = flag(a[6], c.fits) || a[11] != Py_None;
    const auto *pw = c.in<uint16_t>(a[1], at::kBFloat16, {D});
    const auto *pe = res ? c.in<uint16_t>(a[3], at::kBFloat16, {T, D}) : nullptr;
    if (res) c.given(a[7], at::kBFloat16, {T, D});
    else if (a[7] != Py_None) c.fits = false;
    if (y) c.given(a[8], at::kBFloat16, {T, D});
    if (q8) {
        c.given(a[9], at::kChar, {T, D});
        c.given(a[10], at::kFloat, {T});
    }
    c.given(a[11], at::kFloat, {T});
    if (!c.fits) Py_RETURN_NONE;
    Results o(5);
    int8_t *pq = q8 ? c.out<int8_t>(a[9], at::kChar, {T, D}, o.o[0]) : nullptr;
    float *ps = q8 ? c.out<float>(a[10], at::kFloat, {T}, o.o[1]) : nullptr;
    uint16_t *py = y ? c.out<uint16_t>(a[8], at::kBFloat16, {T, D}, o.o[2]) : nullptr;
    uint16_t *ph = res ? c.out<uint16_t>(a[7], at::kBFloat16, {T, D}, o.o[3]) : nullptr;
    float *pr = r ? c.out<float>(a[11], at::kFloat, {T}, o.o[4]) : nullptr;
    const auto *px = static_cast<const uint16_t *>(x->data_ptr());
    void *st = c.stream();
    return o.take(unlocked([&] { return lib.rmsnorm(px, pe, pw, T, D, eps, ph, py, pq, ps, pr, st); }));
    END_HANDLE_TH_ERRORS
}

// rmsnorm_bwd(dY, H, w, rstd, dres, dH, dw) -> (dH, dw)
PyObject *rmsnorm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *dy = n == 7 ? plain(a[0], at::kBFloat16, 2) : nullptr;
    Call c(dy);
    if (!c.fits) Py_RETURN_NONE;
    const int64_t T = dy->size(0), D = dy->size(1);
    const auto *ph = c.in<uint16_t>(a[1], at::kBFloat16, {T, D});
    const auto *pw = c.in<uint16_t>(a[2], at::kBFloat16, {D});
    const auto *pr = c.in<float>(a[3], at::kFloat, {T});
    const auto *pe = a[4] != Py_None ? c.in<uint16_t>(a[4], at::kBFloat16, {T, D}) : nullptr;
    c.given(a[5], at::kBFloat16, {T, D});
    c.given(a[6], at::kFloat, {D});
    int64_t floats = 0;
    if (!c.fits || lib.rmsnorm_bwd_ws(T, D, &floats) != 0) Py_RETURN_NONE;
    Results o(2);
    uint16_t *pdh = c.out<uint16_t>(a[5], at::kBFloat16, {T, D}, o.o[0]);
    float *pdw = c.out<float>(a[6], at::kFloat, {D}, o.o[1]);
    at::Tensor ws;  // its memory may go to a later allocation of this stream, which runs after this call
    if (floats > 0) ws = c.fresh(at::kFloat, {floats});
    float *pws = floats > 0 ? static_cast<float *>(ws.data_ptr()) : nullptr;
    const auto *pdy = static_cast<const uint16_t *>(dy->data_ptr());
    void *st = c.stream();
    return o.take(unlocked([&] { return lib.rmsnorm_bwd(pdy, ph, pw, pr, pe, T, D, pdh, pdw, pws, floats, st); }));
    END_HANDLE_TH_ERRORS
}

// quant_rows(A, Q, scale) -> (Q, scale)
PyObject *quant_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *x = n == 3 ? plain(a[0], at::kBFloat16, 2) : nullptr;
    Call c(x);
    if (!c.fits) Py_RETURN_NONE;
    const int64_t rows = x->size(0), K = x->size(1);
    c.given(a[1], at::kChar, {rows, K});
    c.given(a[2], at::kFloat, {rows});
    if (!c.fits) Py_RETURN_NONE;
    Results o(2);
    int8_t *pq = c.out<int8_t>(a[1], at::kChar, {rows, K}, o.o[0]);
    float *ps = c.out<float>(a[2], at::kFloat, {rows}, o.o[1]);
    const auto *px = static_cast<const uint16_t *>(x->data_ptr());
    void *st = c.stream();
    return o.take(unlocked([&] { return lib.quant_rows(px, rows, K, pq, ps, st); }));
    END_HANDLE_TH_ERRORS
}

// fwd_q8(Xq, xscale, vals_q, wscale, meta, XL, R, out_features, Y) -> Y
PyObject *fwd_q8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t out;
    const at::Tensor *x = n == 9 ? plain(a[0], at::kChar, 2) : nullptr;
    Call c(x);
    if (!c.fits || !as_int(a[7], out)) Py_RETURN_NONE;
    const int64_t T = x->size(0), K = x->size(1);
    const auto *pxs = c.in<float>(a[1], at::kFloat, {T});
    const auto *pv = c.in<int8_t>(a[2], at::kChar, {out, K / 2});
    const auto *pws = c.in<float>(a[3], at::kFloat, {out});
    const auto *pm = c.in<uint16_t>(a[4], at::kShort, {out, K / 16});
    int64_t r = 0;
    const uint16_t *pxl = nullptr, *pr = nullptr;
    if (a[6] != Py_None) {
        const at::Tensor *R = plain(a[6], at::kBFloat16, 2);
        r = R ? R->size(0) : 0;
        pr = c.in<uint16_t>(a[6], at::kBFloat16, {r, out});
        pxl = c.in<uint16_t>(a[5], at::kBFloat16, {T, r});
    } else if (a[5] != Py_None) {
        c.fits = false;
    }
    c.given(a[8], at::kBFloat16, {T, out});
    if (!c.fits) Py_RETURN_NONE;
    Results o(1);
    uint16_t *py = c.out<uint16_t>(a[8], at::kBFloat16, {T, out}, o.o[0]);
    const auto *px = static_cast<const int8_t *>(x->data_ptr());
    void *st = c.stream();
    return o.take(unlocked([&] { return lib.fwd_q8(px, pxs, pv, pws, pm, pxl, pr, T, K, out, r, py, st); }));
    END_HANDLE_TH_ERRORS
}

// bind(addresses): those of rmsnorm, rmsnorm_bwd, rmsnorm_bwd_ws, quant_rows and fwd_q8 in the loaded library
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[5];
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
        return nullptr;
    }
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: NULL address");
            return nullptr;
        }
    }
    lib.rmsnorm = reinterpret_cast<decltype(lib.rmsnorm)>(p[0]);
    lib.rmsnorm_bwd = reinterpret_cast<decltype(lib.rmsnorm_bwd)>(p[1]);
    lib.rmsnorm_bwd_ws = reinterpret_cast<decltype(lib.rmsnorm_bwd_ws)>(p[2]);
    lib.quant_rows = reinterpret_cast<decltype(lib.quant_rows)>(p[3]);
    lib.fwd_q8 = reinterpret_cast<decltype(lib.fwd_q8)>(p[4]);
    Py_RETURN_NONE;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(rmsnorm), METHOD(rmsnorm_bwd), METHOD(quant_rows), METHOD(fwd_q8), {}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
