// torch_bind.cpp -- the quick Python binding of the mixture-of-experts and 4-bit
// entry points: tensors become dg_views on the C++ side, the stream is torch's
// current one unless given.  A decoding step makes many calls of a few
// microseconds each; describing five tensors through ctypes costs 7 us of host
// time a call, here it is well under one.
#include <Python.h>

#include <cstring>

#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "dg.h"

namespace {

// One argument as a view; None is a null view.  False: a Python error is set.
struct Arg {
    dg_view v;
    const dg_view *p = nullptr;

    bool set(PyObject *o) {
        if (o == Py_None) return true;
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
            return false;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        switch (t.scalar_type()) {
        case at::kFloat: v.dtype = DG_F32; break;
        case at::kHalf: v.dtype = DG_F16; break;
        case at::kBFloat16: v.dtype = DG_BF16; break;
        case at::kFloat8_e4m3fn: v.dtype = DG_F8E4M3; break;
        case at::kInt: v.dtype = DG_I32; break;
        case at::kLong: v.dtype = DG_I64; break;
        case at::kByte: v.dtype = DG_U8; break;
        default:
            PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
            return false;
        }
        const int64_t nd = t.dim(), es = (int64_t)t.element_size();
        if (nd > 4) {
            PyErr_SetString(PyExc_ValueError, "views have at most 4 dims");
            return false;
        }
        v.ptr = t.data_ptr();
        v.ndim = nd > 0 ? (int32_t)nd : 1;
        v.shape[0] = 1;
        v.stride[0] = es;
        for (int64_t d = 0; d < nd; ++d) {
            v.shape[d] = t.size(d);
            v.stride[d] = t.stride(d) * es;
        }
        p = &v;
        return true;
    }
};

bool to_int(PyObject *o, int32_t *x) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "integer argument out of range");
        return false;
    }
    *x = (int32_t)v;
    return true;
}

// None: the current stream of the current device.
bool to_stream(PyObject *o, hipStream_t *s) {
    if (o == Py_None) {
        *s = c10::hip::getCurrentHIPStream().stream();
        return true;
    }
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) return false;
    *s = static_cast<hipStream_t>(p);
    return true;
}

bool count(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return got == want;
}

// Every wrapper returns the dg_status as an int.  C++ exceptions (torch may
// throw on a tensor without storage, or where no device is present) become
// Python errors.
template <class F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// The call without the interpreter's lock (a launch waits when the queue is full).
template <class F>
PyObject *status(F f) {
    dg_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

PyObject *sort(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Arg ids, off, ord, pos;
        int32_t E;
        hipStream_t s;
        if (!count(n, 6) || !ids.set(a[0]) || !to_int(a[1], &E) || !off.set(a[2]) || !ord.set(a[3]) || !pos.set(a[4]) ||
            !to_stream(a[5], &s))
            return nullptr;
        return status([&] { return dg_moe_sort(ids.p, E, off.p, ord.p, pos.p, s); });
    });
}

PyObject *gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Arg X, ord, Xs;
        int32_t k;
        hipStream_t s;
        if (!count(n, 5) || !X.set(a[0]) || !ord.set(a[1]) || !to_int(a[2], &k) || !Xs.set(a[3]) || !to_stream(a[4], &s))
            return nullptr;
        return status([&] { return dg_moe_gather(X.p, ord.p, k, Xs.p, s); });
    });
}

PyObject *combine(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Arg Ys, pos, w, Y;
        hipStream_t s;
        if (!count(n, 5) || !Ys.set(a[0]) || !pos.set(a[1]) || !w.set(a[2]) || !Y.set(a[3]) || !to_stream(a[4], &s))
            return nullptr;
        return status([&] { return dg_moe_combine(Ys.p, pos.p, w.p, Y.p, s); });
    });
}

PyObject *combine_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Arg dY, Ys, pos, w, dYs, dw;
        hipStream_t s;
        if (!count(n, 7) || !dY.set(a[0]) || !Ys.set(a[1]) || !pos.set(a[2]) || !w.set(a[3]) || !dYs.set(a[4]) ||
            !dw.set(a[5]) || !to_stream(a[6], &s))
            return nullptr;
        return status([&] { return dg_moe_combine_grad(dY.p, Ys.p, pos.p, w.p, dYs.p, dw.p, s); });
    });
}

PyObject *gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Arg A, off, W, C;
        int32_t act;
        hipStream_t s;
        if (!count(n, 6) || !A.set(a[0]) || !off.set(a[1]) || !W.set(a[2]) || !C.set(a[3]) || !to_int(a[4], &act) ||
            !to_stream(a[5], &s))
            return nullptr;
        return status([&] { return dg_moe_gemm(A.p, off.p, W.p, C.p, (dg_act)act, s); });
    });
}

PyObject *gemm_wgrad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Arg A, D, off, dW;
        hipStream_t s;
        if (!count(n, 5) || !A.set(a[0]) || !D.set(a[1]) || !off.set(a[2]) || !dW.set(a[3]) || !to_stream(a[4], &s))
            return nullptr;
        return status([&] { return dg_moe_gemm_wgrad(A.p, D.p, off.p, dW.p, s); });
    });
}

PyObject *w4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Arg A, Q, S, Z, C;
        int32_t group, act;
        hipStream_t s;
        if (!count(n, 8) || !A.set(a[0]) || !Q.set(a[1]) || !S.set(a[2]) || !Z.set(a[3]) || !C.set(a[4]) ||
            !to_int(a[5], &group) || !to_int(a[6], &act) || !to_stream(a[7], &s))
            return nullptr;
        return status([&] { return dg_gemm_w4(A.p, Q.p, S.p, Z.p, C.p, group, (dg_act)act, s); });
    });
}

PyObject *moe_w4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Arg A, off, Q, S, Z, C;
        int32_t group, act;
        hipStream_t s;
        if (!count(n, 9) || !A.set(a[0]) || !off.set(a[1]) || !Q.set(a[2]) || !S.set(a[3]) || !Z.set(a[4]) ||
            !C.set(a[5]) || !to_int(a[6], &group) || !to_int(a[7], &act) || !to_stream(a[8], &s))
            return nullptr;
        return status([&] { return dg_moe_gemm_w4(A.p, off.p, Q.p, S.p, Z.p, C.p, group, (dg_act)act, s); });
    });
}

// The view of a tensor as bytes (the layout of dg_view), for tests.
PyObject *view(PyObject *, PyObject *o) {
    return guarded([&]() -> PyObject * {
        Arg t;
        std::memset(&t.v, 0, sizeof t.v);
        if (!t.set(o)) return nullptr;
        return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(&t.v), sizeof t.v);
    });
}

#define DG_FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    DG_FAST("moe_sort", sort), DG_FAST("moe_gather", gather), DG_FAST("moe_combine", combine),
    DG_FAST("moe_combine_grad", combine_grad), DG_FAST("moe_gemm", gemm), DG_FAST("moe_gemm_wgrad", gemm_wgrad),
    DG_FAST("gemm_w4", w4), DG_FAST("moe_gemm_w4", moe_w4), {"view", view, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dgtorch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dgtorch() { return PyModule_Create(&module); }
