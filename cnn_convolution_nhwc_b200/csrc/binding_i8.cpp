// Short host path of the 8-bit operators' Python binding: takes the tensors as they are, looks at
// their types, shapes, strides and device, and calls the C entry point on the current stream. What
// it does not find in order it leaves alone and returns kAskSlow: the checked wrapper in Python then
// makes the same call, or raises the error that says what is wrong. A single-token call takes 2 to 5
// us on the GPU; through the wrapper and ctypes it takes 8 us on the host, through here 5.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

namespace {

constexpr int kAskSlow = -1000;

using NormFn = int (*)(const void *, const void *, const float *, void *, int8_t *, float *, int, int, int, float, int, void *);
using RowsFn = int (*)(const void *, int8_t *, float *, int, int, int, int, int, void *);
using FilterFn = int (*)(const void *, int8_t *, float *, int, int, int, int, void *);
using DequantFn = int (*)(const int8_t *, const float *, void *, int, int, int, int, void *);
using PointwiseFn = int (*)(const int8_t *, const float *, const int8_t *, const float *, const float *, void *, int, int, int,
                            int, int, int, void *);
using LayerFn = int (*)(const void *, const float *, float, const int8_t *, const float *, const float *, void *, void *, size_t,
                        int, int, int, int, int, int, void *);

NormFn g_norm;
RowsFn g_rows;
FilterFn g_filter;
DequantFn g_dequant;
PointwiseFn g_pointwise;
LayerFn g_layer;

constexpr int64_t kIntMax = 2147483647;

// The arguments of one call; `ok` falls with the first that is not in order.
struct Args {
    bool ok = true;
    int device = -1;

    const at::Tensor *tensor(PyObject *o) {
        if (!ok || !THPVariable_Check(o)) { ok = false; return nullptr; }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.defined() || !t.is_cuda()) { ok = false; return nullptr; }
        const int d = t.get_device();
        if (device < 0) device = d;
        if (d != device) { ok = false; return nullptr; }
        return &t;
    }
    // A contiguous matrix of bfloat16 (type 0) or float32 (type 1).
    void *matrix(PyObject *o, int64_t &rows, int64_t &cols, int &type) {
        const at::Tensor *t = tensor(o);
        if (!t || t->dim() != 2 || !t->is_contiguous()) { ok = false; return nullptr; }
        if (t->scalar_type() == at::kBFloat16) type = 0;
        else if (t->scalar_type() == at::kFloat) type = 1;
        else { ok = false; return nullptr; }
        rows = t->size(0);
        cols = t->size(1);
        if (rows > kIntMax || cols > kIntMax) ok = false;
        return t->data_ptr();
    }
    // The same with a known shape and type.
    void *matrix_like(PyObject *o, int64_t rows, int64_t cols, int type) {
        int64_t r = 0, c = 0;
        int y = 0;
        void *p = matrix(o, r, c, y);
        if (r != rows || c != cols || y != type) ok = false;
        return p;
    }
    // A contiguous bfloat16 image batch; `shape` is set, or with `same` compared.
    void *images(PyObject *o, int64_t (&shape)[4], bool same) {
        const at::Tensor *t = tensor(o);
        if (!t || t->dim() != 4 || t->scalar_type() != at::kBFloat16 || !t->is_contiguous()) { ok = false; return nullptr; }
        for (int i = 0; i < 4; ++i) {
            const int64_t n = t->size(i);
            if (n > kIntMax || (same && n != shape[i])) ok = false;
            shape[i] = n;
        }
        return t->data_ptr();
    }
    float *floats(PyObject *o, int64_t n) {
        const at::Tensor *t = tensor(o);
        if (!t || t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return static_cast<float *>(t->data_ptr());
    }
    // 8-bit rows: contiguous bytes, rows a multiple of 16 bytes apart.
    int8_t *bytes(PyObject *o, int64_t &rows, int64_t &cols, int &ld) {
        const at::Tensor *t = tensor(o);
        if (!t || t->scalar_type() != at::kChar || t->dim() != 2) { ok = false; return nullptr; }
        rows = t->size(0);
        cols = t->size(1);
        const int64_t pitch = rows < 2 ? (cols + 15) / 16 * 16 : t->stride(0);
        if ((cols > 1 && t->stride(1) != 1) || pitch < cols || pitch % 16 != 0 || rows > kIntMax || pitch > kIntMax) {
            ok = false;
            return nullptr;
        }
        ld = static_cast<int>(pitch);
        return static_cast<int8_t *>(t->data_ptr());
    }
    // The current stream, if the tensors are on the current device.
    bool ready(void *&stream) {
        if (!ok || device != c10::cuda::current_device()) return false;
        stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
        return true;
    }
};

template <class F>
PyObject *guarded(F f) {
    int rc = kAskSlow;
    try {
        rc = f();
    } catch (const std::exception &) {
        rc = kAskSlow;   // the checked path meets and reports it
    }
    return PyLong_FromLong(rc);
}

// (x, weight, residual or None, h or None, q, scale, eps)
PyObject *rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> int {
        if (n != 7 || !PyFloat_Check(a[6])) return kAskSlow;
        Args g;
        int64_t M = 0, C = 0, r = 0, c = 0;
        int type = 0, ld = 0;
        const void *x = g.matrix(a[0], M, C, type);
        const float *w = g.floats(a[1], C);
        const void *res = nullptr;
        void *h = nullptr, *stream = nullptr;
        if (a[2] != Py_None) {
            res = g.matrix_like(a[2], M, C, type);
            h = g.matrix_like(a[3], M, C, type);
        } else if (a[3] != Py_None) {
            return kAskSlow;
        }
        int8_t *q = g.bytes(a[4], r, c, ld);
        float *s = g.floats(a[5], M);
        if (!g.ready(stream) || r != M || c != C) return kAskSlow;
        return g_norm(x, res, w, h, q, s, (int)M, (int)C, ld, (float)PyFloat_AS_DOUBLE(a[6]), type, stream);
    });
}

// (x, q, scale, glu)
PyObject *rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> int {
        if (n != 4) return kAskSlow;
        Args g;
        int64_t M = 0, C = 0, r = 0, c = 0;
        int type = 0, ld = 0;
        void *stream = nullptr;
        const void *x = g.matrix(a[0], M, C, type);
        int8_t *q = g.bytes(a[1], r, c, ld);
        float *s = g.floats(a[2], M);
        const int glu = a[3] == Py_True;
        if (!g.ready(stream) || r != M || c * (glu ? 2 : 1) != C) return kAskSlow;
        return g_rows(x, q, s, (int)M, (int)c, ld, glu, type, stream);
    });
}

// (F, q, scale)
PyObject *filter(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> int {
        if (n != 3) return kAskSlow;
        Args g;
        int64_t Cin = 0, Cout = 0, r = 0, c = 0;
        int type = 0, ld = 0;
        void *stream = nullptr;
        const void *f = g.matrix(a[0], Cin, Cout, type);
        int8_t *q = g.bytes(a[1], r, c, ld);
        float *s = g.floats(a[2], Cout);
        if (!g.ready(stream) || r != Cout || c != Cin) return kAskSlow;
        return g_filter(f, q, s, (int)Cin, (int)Cout, ld, type, stream);
    });
}

// (q, scale, y)
PyObject *dequant(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> int {
        if (n != 3) return kAskSlow;
        Args g;
        int64_t M = 0, C = 0, r = 0, c = 0;
        int type = 0, ld = 0;
        void *stream = nullptr;
        const int8_t *q = g.bytes(a[0], M, C, ld);
        const float *s = g.floats(a[1], M);
        void *y = g.matrix(a[2], r, c, type);
        if (!g.ready(stream) || r != M || c != C) return kAskSlow;
        return g_dequant(q, s, y, (int)M, (int)C, ld, type, stream);
    });
}

// (q, q_scale, Wq, w_scale, bias or None, y)
PyObject *pointwise(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> int {
        if (n != 6) return kAskSlow;
        Args g;
        int64_t M = 0, Cin = 0, Cout = 0, c = 0, r = 0, yc = 0;
        int type = 0, ldq = 0, ldw = 0;
        void *stream = nullptr;
        const int8_t *q = g.bytes(a[0], M, Cin, ldq);
        const float *qs = g.floats(a[1], M);
        const int8_t *w = g.bytes(a[2], Cout, c, ldw);
        const float *ws = g.floats(a[3], Cout);
        const float *bias = a[4] == Py_None ? nullptr : g.floats(a[4], Cout);
        void *y = g.matrix(a[5], r, yc, type);
        if (!g.ready(stream) || c != Cin || r != M || yc != Cout) return kAskSlow;
        return g_pointwise(q, qs, w, ws, bias, y, (int)M, (int)Cin, (int)Cout, ldq, ldw, type, stream);
    });
}

// (X, norm or None, eps, Wq, w_scale, bias or None, Y, workspace)
PyObject *layer(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> int {
        if (n != 8 || !PyFloat_Check(a[2])) return kAskSlow;
        Args g;
        int64_t x[4] = {}, Cout = 0, c = 0;
        int ldw = 0;
        void *stream = nullptr;
        const void *X = g.images(a[0], x, false);
        const float *norm = a[1] == Py_None ? nullptr : g.floats(a[1], x[3]);
        const int8_t *w = g.bytes(a[3], Cout, c, ldw);
        const float *ws = g.floats(a[4], Cout);
        const float *bias = a[5] == Py_None ? nullptr : g.floats(a[5], Cout);
        int64_t y[4] = {x[0], x[1], x[2], Cout};
        void *Y = g.images(a[6], y, true);
        const at::Tensor *space = g.tensor(a[7]);
        if (!g.ready(stream) || c != x[3] || !space->is_contiguous()) return kAskSlow;
        return g_layer(X, norm, (float)PyFloat_AS_DOUBLE(a[2]), w, ws, bias, Y, space->data_ptr(), space->nbytes(), (int)x[0],
                       (int)x[1], (int)x[2], (int)x[3], (int)Cout, ldw, stream);
    });
}

// (six addresses: the entry points of the library that the package has loaded)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[6] = {};
    for (Py_ssize_t i = 0; i < n && i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_norm = reinterpret_cast<NormFn>(p[0]);
    g_rows = reinterpret_cast<RowsFn>(p[1]);
    g_filter = reinterpret_cast<FilterFn>(p[2]);
    g_dequant = reinterpret_cast<DequantFn>(p[3]);
    g_pointwise = reinterpret_cast<PointwiseFn>(p[4]);
    g_layer = reinterpret_cast<LayerFn>(p[5]);
    if (!g_norm || !g_rows || !g_filter || !g_dequant || !g_pointwise || !g_layer) {
        PyErr_SetString(PyExc_ValueError, "bind takes six addresses");
        return nullptr;
    }
    Py_RETURN_NONE;
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(bind), ENTRY(rmsnorm), ENTRY(rows), ENTRY(filter), ENTRY(dequant), ENTRY(pointwise), ENTRY(layer),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding_i8", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding_i8() { return PyModule_Create(&g_module); }
