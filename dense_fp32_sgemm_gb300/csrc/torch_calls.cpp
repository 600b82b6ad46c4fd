// The usual calls of the norm and of the operators in 8 bits, from torch tensors straight
// to the C ABI: checks, outputs, stream.
//
// On the host such a call takes 14 to 18 us in Python (Grace), several times as long as
// its kernel on the device, and 5 to 7 here (2 to 4 with outputs given).  What is not usual (another stream or
// device, a gradient to record, other types, shapes or strides, tensor subclasses) gets
// None, and the Python wrapper checks, refuses or does it.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "../../include/sgemm_ffn.h"
#include "../../include/sgemm_q8.h"

namespace {

// SGEMM_TYPE_* of a tensor's type, or -1.
int type_of(at::ScalarType t) {
    return t == at::kFloat ? SGEMM_TYPE_F32 : t == at::kHalf ? SGEMM_TYPE_F16 : t == at::kBFloat16 ? SGEMM_TYPE_BF16 : -1;
}

// An argument: a tensor, or nothing.  `ok` turns false for anything else.
const at::Tensor *tensor(PyObject *o, bool &ok) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_CheckExact(o)) {
        ok = false;
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}

struct Rows {
    void *p = nullptr;
    int64_t ld = 1;
};
// A row-major rows x cols matrix of this type on this device (or none of it).
bool rows_of(const at::Tensor *t, at::ScalarType type, int64_t device, int64_t rows, int64_t cols, Rows &out) {
    out.ld = cols > 1 ? cols : 1;
    if (!t) return true;
    if (!t->is_cuda() || t->get_device() != device || t->scalar_type() != type || t->dim() != 2 ||
        t->size(0) != rows || t->size(1) != cols || (cols > 1 && t->stride(1) != 1) ||
        (rows > 1 && t->stride(0) < cols))
        return false;
    out.p = t->data_ptr();
    if (rows > 1 && t->stride(0) > 1) out.ld = t->stride(0);
    return true;
}
bool vector_of(const at::Tensor *t, at::ScalarType type, int64_t device, int64_t n) {
    return t && t->is_cuda() && t->get_device() == device && t->scalar_type() == type && t->dim() == 1 &&
           t->size(0) == n && t->is_contiguous();
}
// Whether one requires a gradient to be recorded, or carries a tangent of forward-mode
// differentiation (of the one level that there is).
bool wants_graph(std::initializer_list<const at::Tensor *> list) {
    const bool records = at::GradMode::is_enabled();
    for (const at::Tensor *t : list)
        if (t && ((records && t->requires_grad()) || t->_fw_grad(0).defined())) return true;
    return false;
}
// A given output (one that requires a gradient is refused in Python): graphs that hold it will
// know that it was overwritten.
void written(const at::Tensor *t) {
    if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
at::Tensor codes(int64_t rows, int64_t cols, const at::Tensor &like) {
    const int64_t ld = cols > 16 ? (cols + 15) / 16 * 16 : 16;
    return at::empty_strided({rows, cols}, {ld, 1}, like.options().dtype(at::kChar));
}
at::Tensor floats(int64_t n, const at::Tensor &like) { return at::empty({n}, like.options().dtype(at::kFloat)); }

// A new reference to a given output, or to one made here.
PyObject *give(PyObject *given, const at::Tensor &made) {
    if (given != Py_None) {
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(made);
}
PyObject *none() {
    Py_INCREF(Py_None);
    return Py_None;
}
// A tuple of new references, which it takes.
PyObject *pack(std::initializer_list<PyObject *> items) {
    PyObject *t = PyTuple_New((Py_ssize_t)items.size());
    bool ok = t != nullptr;
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        ok = ok && o;
        if (t)
            PyTuple_SET_ITEM(t, i++, o);
        else
            Py_XDECREF(o);
    }
    if (ok) return t;
    Py_XDECREF(t);
    return nullptr;
}

// What a norm's call is about, where it is a usual one.
struct Norm {
    const at::Tensor *x, *weight, *residual;
    at::ScalarType kind;
    int type, weight_type;
    int64_t device, T, D;
    Rows xr, rr;
    double eps;
    void *stream;

    bool usual(PyObject *px, PyObject *pw, PyObject *pr, PyObject *peps) {
        bool ok = true;
        x = tensor(px, ok);
        weight = tensor(pw, ok);
        residual = tensor(pr, ok);
        if (!ok || !x || !weight || !x->is_cuda() || x->dim() != 2) return false;
        eps = PyFloat_CheckExact(peps) ? PyFloat_AS_DOUBLE(peps) : -1.0;
        kind = x->scalar_type();
        type = type_of(kind);
        weight_type = type_of(weight->scalar_type());
        device = x->get_device();
        T = x->size(0);
        D = x->size(1);
        if (!(eps >= 0.0) || type < 0 || (weight_type != type && weight_type != SGEMM_TYPE_F32) ||
            device != c10::cuda::current_device() || !rows_of(x, kind, device, T, D, xr) ||
            !rows_of(residual, kind, device, T, D, rr) || !vector_of(weight, weight->scalar_type(), device, D))
            return false;
        stream = c10::cuda::getCurrentCUDAStream(device).stream();
        return true;
    }
    at::Tensor empty() const { return at::empty({T, D}, x->options()); }
};

// Runs a call without the interpreter's lock; a status other than 0 becomes a number.
template <class Call>
PyObject *failed(Call &&call) {
    sgemm_status_t s;
    Py_BEGIN_ALLOW_THREADS
    s = call();
    Py_END_ALLOW_THREADS
    return s == SGEMM_OK ? nullptr : PyLong_FromLong(s);
}

// rms_norm(x, weight, residual, eps, y, h) -> y, (y, h), None or a status.
PyObject *rms_norm(PyObject *const *a) {
    Norm n;
    bool ok = n.usual(a[0], a[1], a[2], a[3]);
    if (!ok) Py_RETURN_NONE;
    const at::Tensor *y = tensor(a[4], ok), *h = tensor(a[5], ok);
    Rows yr, hr;
    if (!ok || wants_graph({n.x, n.weight, n.residual, y, h}) || !rows_of(y, n.kind, n.device, n.T, n.D, yr) ||
        !rows_of(h, n.kind, n.device, n.T, n.D, hr) || (yr.p && yr.p == hr.p))
        Py_RETURN_NONE;
    at::Tensor new_y, new_h;
    if (!y) {
        new_y = n.empty();
        yr.p = new_y.data_ptr();
    }
    if (!h && n.residual) {
        new_h = n.empty();
        hr.p = new_h.data_ptr();
    }
    written(y);
    written(h);
    PyObject *f = failed([&] {
        return sgemm_rms_norm(n.T, n.D, n.type, n.xr.p, n.xr.ld, n.rr.p, n.rr.ld, n.weight->data_ptr(), n.weight_type,
                              n.eps, hr.p, hr.ld, yr.p, yr.ld, n.stream);
    });
    if (f) return f;
    if (!n.residual) return give(a[4], new_y);
    return pack({give(a[4], new_y), give(a[5], new_h)});
}

// rms_norm_q8(x, weight, residual, eps, h) -> (q, scales), (q, scales, h), None or a status.
PyObject *rms_norm_q8(PyObject *const *a) {
    Norm n;
    bool ok = n.usual(a[0], a[1], a[2], a[3]);
    if (!ok) Py_RETURN_NONE;
    const at::Tensor *h = tensor(a[4], ok);
    Rows hr;
    if (!ok || wants_graph({n.x, n.weight, n.residual, h}) || !rows_of(h, n.kind, n.device, n.T, n.D, hr))
        Py_RETURN_NONE;
    at::Tensor new_h;
    if (!h && n.residual) {
        new_h = n.empty();
        hr.p = new_h.data_ptr();
    }
    written(h);
    const at::Tensor q = codes(n.T, n.D, *n.x), scales = floats(n.T, *n.x);
    PyObject *f = failed([&] {
        return sgemm_rms_norm_q8(n.T, n.D, n.type, n.xr.p, n.xr.ld, n.rr.p, n.rr.ld, n.weight->data_ptr(),
                                 n.weight_type, n.eps, hr.p, hr.ld, static_cast<int8_t *>(q.data_ptr()),
                                 n.D > 16 ? (n.D + 15) / 16 * 16 : 16, static_cast<float *>(scales.data_ptr()), n.stream);
    });
    if (f) return f;
    if (!n.residual) return pack({THPVariable_Wrap(q), THPVariable_Wrap(scales)});
    return pack({THPVariable_Wrap(q), THPVariable_Wrap(scales), give(a[4], new_h)});
}

// rms_norm_backward(x, weight, residual, eps, dy, dh, dx, dweight, need_dx, need_dw)
// -> (dx, dweight), None or a status.
PyObject *rms_norm_backward(PyObject *const *a) {
    Norm n;
    bool ok = n.usual(a[0], a[1], a[2], a[3]);
    if (!ok) Py_RETURN_NONE;
    const bool need_dx = a[8] == Py_True, need_dw = a[9] == Py_True;
    const at::Tensor *dy = tensor(a[4], ok), *dh = tensor(a[5], ok), *dx = tensor(a[6], ok), *dw = tensor(a[7], ok);
    Rows dyr, dhr, dxr;
    if (!ok || !dy || wants_graph({n.x, n.weight, n.residual, dy, dh, need_dx ? dx : nullptr, need_dw ? dw : nullptr}) ||
        !rows_of(dy, n.kind, n.device, n.T, n.D, dyr) || !rows_of(dh, n.kind, n.device, n.T, n.D, dhr) ||
        (need_dx && !rows_of(dx, n.kind, n.device, n.T, n.D, dxr)) ||
        (need_dw && dw && !vector_of(dw, n.weight->scalar_type(), n.device, n.D)) ||
        (a[8] != Py_True && a[8] != Py_False) || (a[9] != Py_True && a[9] != Py_False))
        Py_RETURN_NONE;
    at::Tensor new_dx, new_dw;
    if (need_dx && !dx) {
        new_dx = n.empty();
        dxr.p = new_dx.data_ptr();
    }
    if (need_dw && !dw) new_dw = at::empty({n.D}, n.weight->options());
    if (need_dx) written(dx);
    if (need_dw) written(dw);
    void *dwp = !need_dw ? nullptr : dw ? dw->data_ptr() : new_dw.data_ptr();
    PyObject *f = failed([&] {
        return sgemm_rms_norm_backward(n.T, n.D, n.type, n.xr.p, n.xr.ld, n.rr.p, n.rr.ld, n.weight->data_ptr(),
                                       n.weight_type, n.eps, dyr.p, dyr.ld, dhr.p, dhr.ld, need_dx ? dxr.p : nullptr,
                                       dxr.ld, dwp, n.stream);
    });
    if (f) return f;
    return pack({need_dx ? give(a[6], new_dx) : none(), need_dw ? give(a[7], new_dw) : none()});
}

// gate_q8(g, u or None, activation) -> (q, scales), None or a status.
PyObject *gate_q8(PyObject *const *a) {
    bool ok = true;
    const at::Tensor *g = tensor(a[0], ok), *u = tensor(a[1], ok);
    if (!ok || !g || !g->is_cuda() || g->dim() != 2 || !PyLong_CheckExact(a[2]) || wants_graph({g, u})) Py_RETURN_NONE;
    const long act = PyLong_AsLong(a[2]);
    const int type = type_of(g->scalar_type());
    const int64_t device = g->get_device(), T = g->size(0), F = g->size(1);
    Rows gr, ur;
    if (PyErr_Occurred() || act < 0 || act > 1000 || type < 0 || device != c10::cuda::current_device() ||
        !rows_of(g, g->scalar_type(), device, T, F, gr) || !rows_of(u, g->scalar_type(), device, T, F, ur)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const at::Tensor q = codes(T, F, *g), scales = floats(T, *g);
    void *stream = c10::cuda::getCurrentCUDAStream(device).stream();
    PyObject *f = failed([&] {
        return sgemm_q8_gate(T, F, type, (int)act, gr.p, gr.ld, ur.p, ur.ld, static_cast<int8_t *>(q.data_ptr()),
                             F > 16 ? (F + 15) / 16 * 16 : 16, static_cast<float *>(scales.data_ptr()), stream);
    });
    if (f) return f;
    return pack({THPVariable_Wrap(q), THPVariable_Wrap(scales)});
}

// q8_matmul(x, x_scales, y, (N, K, type, w, ldw, w_scales, device)) -> y, None or a status.
PyObject *q8_matmul(PyObject *const *a) {
    bool ok = true;
    const at::Tensor *x = tensor(a[0], ok), *xs = tensor(a[1], ok), *y = tensor(a[2], ok);
    if (!ok || !x || !xs || !x->is_cuda() || x->dim() != 2 || !PyTuple_CheckExact(a[3]) || PyTuple_GET_SIZE(a[3]) != 7 ||
        wants_graph({xs, y}))
        Py_RETURN_NONE;
    long long m[7];
    for (int i = 0; i < 7; ++i) m[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(a[3], i));
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const int64_t N = m[0], K = m[1], M = x->size(0), device = m[6];
    const at::ScalarType kind = m[2] == SGEMM_TYPE_F32 ? at::kFloat : m[2] == SGEMM_TYPE_F16 ? at::kHalf : at::kBFloat16;
    Rows xr, yr;
    if (device != c10::cuda::current_device() || !rows_of(x, at::kChar, device, M, K, xr) ||
        !vector_of(xs, at::kFloat, device, M) || !rows_of(y, kind, device, M, N, yr))
        Py_RETURN_NONE;
    at::Tensor new_y;
    if (!y) {
        new_y = at::empty({M, N}, x->options().dtype(kind));
        yr.p = new_y.data_ptr();
    }
    written(y);
    void *stream = c10::cuda::getCurrentCUDAStream(device).stream();
    PyObject *f = failed([&] {
        return sgemm_q8_matmul(M, N, K, (int)m[2], static_cast<const int8_t *>(xr.p), xr.ld,
                               static_cast<const float *>(xs->data_ptr()), reinterpret_cast<const int8_t *>(m[3]), m[4],
                               reinterpret_cast<const float *>(m[5]), yr.p, yr.ld, stream);
    });
    return f ? f : give(a[2], new_y);
}

// A Python function of `N` positional arguments; C++ exceptions become Python's.
template <PyObject *(*CALL)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t count) {
    if (count != N) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return CALL(args);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}
template <PyObject *(*CALL)(PyObject *const *), int N>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<CALL, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rms_norm, 6>("rms_norm"), method<rms_norm_q8, 5>("rms_norm_q8"),
                         method<rms_norm_backward, 10>("rms_norm_backward"), method<gate_q8, 3>("gate_q8"),
                         method<q8_matmul, 4>("q8_matmul"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__torch_calls() { return PyModule_Create(&module); }
