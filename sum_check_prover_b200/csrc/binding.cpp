// The binding's short way for the layer operators: a decode step makes several calls of a few microseconds, of
// which the interpreter's checks of five tensors and the conversion of a dozen arguments took half (us a call, the
// methods' way and this one: quantised rows 5.4 and 2.4, combine 7.2 and 2.1, gradients 8.1 and 2.5).
//
// Each function here takes what the method of the same name takes, reads the tensors' addresses, sizes and pitches
// directly and makes the C call; it returns the call's status. Whatever it does not know for sure to be right
// (another type, shape, device or layout, an argument that is no tensor) it returns None for, and the method goes
// on to its own checks, which say what is wrong. So nothing is refused or defined here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/fp.h"

namespace {

struct Call {
    fp_ctx* ctx;
    int device;
    void* stream;
};

// the context's handle and device, and the stream: its handle, an object that has one, or None for the device's
// current one
bool call_of(PyObject* handle, PyObject* device, PyObject* stream, Call& c) {
    if (!PyLong_CheckExact(handle) || !PyLong_CheckExact(device)) return false;
    c.ctx = (fp_ctx*)PyLong_AsVoidPtr(handle);
    c.device = (int)PyLong_AsLong(device);
    if (!c.ctx || PyErr_Occurred()) return false;
    if (stream == Py_None) {
        c.stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c.device).stream();
        return true;
    }
    PyObject* own = PyLong_CheckExact(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
    if (!own) return false;
    const bool number = PyLong_CheckExact(own);
    if (number) c.stream = PyLong_AsVoidPtr(own);
    Py_DECREF(own);
    return number && !PyErr_Occurred();
}

// a plain tensor (no subclass, no wrapper, nothing still to be conjugated or negated) on the context's device
const at::Tensor* tensor_of(PyObject* o, const Call& c, int64_t dims) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    const bool plain = t.defined() && t.layout() == at::kStrided && t.is_cuda() && !t.is_conj() && !t.is_neg();
    return plain && t.get_device() == c.device && t.dim() == dims ? &t : nullptr;
}

struct Rows {
    void* p;
    int64_t n, m, ld;
    at::ScalarType type;
};

// a matrix whose rows may be part of wider ones
bool rows_of(PyObject* o, const Call& c, Rows& r) {
    const at::Tensor* t = tensor_of(o, c, 2);
    if (!t) return false;
    r.n = t->size(0), r.m = t->size(1), r.type = t->scalar_type();
    const int64_t ld = t->stride(0);
    if ((r.m > 1 && t->stride(1) != 1) || (r.n > 1 && ld < r.m)) return false;
    r.ld = r.n > 1 ? ld : r.m;
    r.p = t->mutable_data_ptr();
    return true;
}

// a contiguous tensor of a given type; sizes of up to three dimensions, -1 for any
bool dense_of(PyObject* o, const Call& c, at::ScalarType type, int64_t dims, const int64_t* size, void*& p) {
    const at::Tensor* t = tensor_of(o, c, dims);
    if (!t || t->scalar_type() != type || !t->is_contiguous()) return false;
    for (int64_t i = 0; i < dims; i++)
        if (size[i] >= 0 && t->size(i) != size[i]) return false;
    p = t->mutable_data_ptr();
    return true;
}

// T x k positions
bool positions_of(PyObject* o, const Call& c, int64_t T, void*& p, int64_t& k) {
    const int64_t size[2] = {T, -1};
    if (!dense_of(o, c, at::kInt, 2, size, p)) return false;
    k = THPVariable_Unpack(o).size(1);
    return k <= INT32_MAX;
}

int real_of(at::ScalarType t) {
    return t == at::kFloat ? FP_F32 : t == at::kHalf ? FP_F16 : t == at::kBFloat16 ? FP_BF16 : -1;
}

// The interpreter's lock is free during the C call, as in a call through ctypes: a launch may wait for room in its
// stream's queue.
template <class F> PyObject* status_of(F&& call) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

// One function of the module: the status, or None when `run` returns null. No exception crosses into the interpreter,
// C++'s or its own.
template <PyObject* (*run)(PyObject* const*), int N> PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    PyObject* rc = nullptr;
    try {
        if (n == N) rc = run(a);
    } catch (const std::exception&) {
    }
    if (rc) return rc;
    PyErr_Clear();
    Py_RETURN_NONE;
}

// quantize_rows(handle, device, x, q, scale, pos, stream)
PyObject* quantize_rows(PyObject* const* a) {
    Call c;
    Rows x, q;
    void *scale, *pos = nullptr;
    int64_t k = 0;
    if (!call_of(a[0], a[1], a[6], c) || !rows_of(a[2], c, x) || !rows_of(a[3], c, q)) return nullptr;
    const int type = real_of(x.type);
    if (type < 0 || q.type != at::kChar || q.m != x.m || !dense_of(a[4], c, at::kFloat, 1, &q.n, scale)) return nullptr;
    if (a[5] != Py_None && !positions_of(a[5], c, x.n, pos, k)) return nullptr;
    return status_of([&] {
        return fp_quantize_rows(c.ctx, x.p, type, x.n, x.m, x.ld, (const int32_t*)pos, (int)k, q.n, (int8_t*)q.p,
                                q.ld, (float*)scale, c.stream);
    });
}

// matmul_i8(handle, device, w, x, y, w_scale, x_scale, offsets, stream)
PyObject* matmul_i8(PyObject* const* a) {
    Call c;
    Rows w, x, y;
    void *ws, *xs, *off = nullptr;
    int64_t E = 1;
    if (!call_of(a[0], a[1], a[8], c) || !rows_of(a[3], c, x) || !rows_of(a[4], c, y)) return nullptr;
    if (a[7] == Py_None) {
        if (!rows_of(a[2], c, w) || !dense_of(a[5], c, at::kFloat, 1, &w.n, ws)) return nullptr;
    } else {
        const int64_t any[3] = {-1, -1, -1};
        if (!dense_of(a[2], c, at::kChar, 3, any, w.p)) return nullptr;
        const at::Tensor& t = THPVariable_Unpack(a[2]);
        E = t.size(0), w.n = t.size(1), w.m = w.ld = t.size(2), w.type = at::kChar;
        const int64_t size[2] = {E, w.n}, ends = E + 1;
        if (!dense_of(a[5], c, at::kFloat, 2, size, ws) || !dense_of(a[7], c, at::kInt, 1, &ends, off)) return nullptr;
    }
    const int type = real_of(y.type);
    if (type < 0 || w.type != at::kChar || x.type != at::kChar || x.m != w.m || y.n != x.n || y.m != w.n || E > INT32_MAX ||
        !dense_of(a[6], c, at::kFloat, 1, &x.n, xs))
        return nullptr;
    return status_of([&] {
        return fp_matmul_i8(c.ctx, (const int8_t*)w.p, w.ld, (const float*)ws, (int)E, w.n, w.m, (const int8_t*)x.p,
                            x.ld, (const float*)xs, x.n, (const int32_t*)off, y.p, type, y.ld, c.stream);
    });
}

// moe_sort(handle, device, e, E, offsets, pos, stream)
PyObject* moe_sort(PyObject* const* a) {
    Call c;
    if (!call_of(a[0], a[1], a[6], c) || !PyLong_CheckExact(a[3]) || !THPVariable_CheckExact(a[2])) return nullptr;
    const int64_t E = PyLong_AsLongLong(a[3]);
    if (PyErr_Occurred() || E < 1 || E >= INT32_MAX) return nullptr;
    const int64_t ends = E + 1;
    const at::Tensor& t = THPVariable_Unpack(a[2]);
    void *e, *off, *pos;
    if (!t.defined() || !dense_of(a[2], c, at::kInt, t.dim(), t.sizes().data(), e) ||
        !dense_of(a[5], c, at::kInt, t.dim(), t.sizes().data(), pos) || !dense_of(a[4], c, at::kInt, 1, &ends, off))
        return nullptr;
    return status_of([&] {
        return fp_moe_sort(c.ctx, (const int32_t*)e, t.numel(), (int)E, (int32_t*)off, (int32_t*)pos, c.stream);
    });
}

// moe_dispatch(handle, device, x, pos, rows, stream)
PyObject* moe_dispatch(PyObject* const* a) {
    Call c;
    Rows x, r;
    void* pos;
    int64_t k;
    if (!call_of(a[0], a[1], a[5], c) || !rows_of(a[2], c, x) || !rows_of(a[4], c, r) || r.type != x.type || r.m != x.m ||
        !positions_of(a[3], c, x.n, pos, k))
        return nullptr;
    const int64_t size = (int64_t)c10::elementSize(x.type);
    return status_of([&] {
        return fp_moe_dispatch(c.ctx, x.p, x.n, x.m * size, x.ld * size, (const int32_t*)pos, (int)k, r.n, r.p,
                               r.ld * size, c.stream);
    });
}

// moe_combine(handle, device, rows, pos, out, weights, base, stream)
PyObject* moe_combine(PyObject* const* a) {
    Call c;
    Rows r, o, b = {};
    void *pos, *w = nullptr;
    int64_t k;
    if (!call_of(a[0], a[1], a[7], c) || !rows_of(a[2], c, r) || !rows_of(a[4], c, o) || o.m != r.m ||
        !positions_of(a[3], c, o.n, pos, k))
        return nullptr;
    const int64_t size[2] = {o.n, k};
    const int rt = real_of(r.type), ot = real_of(o.type);
    if (rt < 0 || ot < 0 || (a[5] != Py_None && !dense_of(a[5], c, at::kFloat, 2, size, w))) return nullptr;
    if (a[6] != Py_None && (!rows_of(a[6], c, b) || b.n != o.n || b.m != o.m || b.type != o.type)) return nullptr;
    return status_of([&] {
        return fp_moe_combine(c.ctx, r.p, rt, r.n, r.ld, (const int32_t*)pos, (const float*)w, b.p, b.ld, o.n, (int)k,
                              o.m, o.p, ot, o.ld, c.stream);
    });
}

// moe_combine_grad(handle, device, dout, rows, pos, weights, drows, dweights, stream)
PyObject* moe_combine_grad(PyObject* const* a) {
    Call c;
    Rows d, r, g = {};
    void *pos, *w = nullptr, *dw = nullptr;
    int64_t k;
    if (!call_of(a[0], a[1], a[8], c) || !rows_of(a[2], c, d) || !rows_of(a[3], c, r) || r.m != d.m ||
        !positions_of(a[4], c, d.n, pos, k))
        return nullptr;
    const int64_t size[2] = {d.n, k};
    const int dt = real_of(d.type), rt = real_of(r.type);
    if (dt < 0 || rt < 0 || (a[5] != Py_None && !dense_of(a[5], c, at::kFloat, 2, size, w)) ||
        (a[7] != Py_None && !dense_of(a[7], c, at::kFloat, 2, size, dw)))
        return nullptr;
    if (a[6] != Py_None && (!rows_of(a[6], c, g) || g.n != r.n || g.m != r.m || g.type != r.type)) return nullptr;
    return status_of([&] {
        return fp_moe_combine_grad(c.ctx, d.p, dt, d.ld, r.p, rt, r.n, r.ld, (const int32_t*)pos, (const float*)w,
                                   d.n, (int)k, d.m, g.p, g.ld, (float*)dw, c.stream);
    });
}

#define FP_ENTRY(name, arguments) {#name, (PyCFunction)(void (*)(void))entry<name, arguments>, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FP_ENTRY(quantize_rows, 7),     FP_ENTRY(matmul_i8, 9),   FP_ENTRY(moe_sort, 7),
                          FP_ENTRY(moe_dispatch, 6),      FP_ENTRY(moe_combine, 8), FP_ENTRY(moe_combine_grad, 9),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch: the version of PyTorch that this was compiled against, whose tensors' layout it relies on
PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&kModule);
    if (m && PyModule_AddStringConstant(m, "torch", FP_TORCH) != 0) Py_CLEAR(m);
    return m;
}
