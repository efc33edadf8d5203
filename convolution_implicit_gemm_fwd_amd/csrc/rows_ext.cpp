// rows_ext.cpp -- the row operators' calls from torch in their common case:
// tensors on the current device and stream, contiguous or two-dimensional
// rows, every argument as it should be.  Each function takes the arguments of
// the Python function of its name (without the stream), allocates the outputs
// and the workspace, calls the C ABI and returns the tensors; for anything
// else it returns None and does nothing, and the Python function checks,
// reports or handles it.
//
// A small call's time is the host's: one token's layer norm takes it 4.3 us
// here and 7.0 in Python (an allocation 0.4 instead of 1.2, the checks and the
// call 0.5 instead of 2.5), of which the launch is 3.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "convimg.h"

namespace {

// The C ABI, bound by address from the library that the package has loaded.
decltype(&layer_norm_fwd) p_layer_norm_fwd;
decltype(&layer_norm_fwd_mxfp4) p_layer_norm_fwd_mxfp4;
decltype(&layer_norm_bwd) p_layer_norm_bwd;
decltype(&layer_norm_bwd_workspace) p_layer_norm_bwd_workspace;
decltype(&mxfp4_quantize) p_mxfp4_quantize;
decltype(&mxfp4_dequantize) p_mxfp4_dequantize;
decltype(&mxfp4_linear_fwd) p_mxfp4_linear_fwd;
decltype(&mxfp4_linear_workspace) p_mxfp4_linear_workspace;
decltype(&mxfp4_linear_bwd) p_mxfp4_linear_bwd;
decltype(&mxfp4_linear_bwd_workspace) p_mxfp4_linear_bwd_workspace;

int type_code(at::ScalarType t)
{
    switch (t) {
    case at::kBFloat16: return CONVIMG_BF16;
    case at::kFloat: return CONVIMG_FP32;
    case at::kHalf: return CONVIMG_FP16;
    default: return -1;
    }
}

// The scalar type of a dtype object, or `other` for None.
bool type_of(PyObject *o, at::ScalarType other, at::ScalarType &t)
{
    if (o == Py_None)
        t = other;
    else if (THPDtype_Check(o))
        t = reinterpret_cast<THPDtype *>(o)->scalar_type;
    else
        return false;
    return type_code(t) >= 0;
}

bool tensor_of(PyObject *o, const at::Tensor *&t)
{
    if (!THPVariable_CheckExact(o))
        return false;
    t = &THPVariable_Unpack(o);
    return t->is_cuda() && t->layout() == at::kStrided && t->device().index() == c10::hip::current_device();
}

// Rows of one of the three types: contiguous, or two-dimensional with
// contiguous columns.
struct Rows {
    const at::Tensor *t = nullptr;
    void *p = nullptr;
    int64_t rows = 0, ld = 0;
    int cols = 0, type = -1;

    bool of(PyObject *o)
    {
        if (!tensor_of(o, t))
            return false;
        const auto sizes = t->sizes(), strides = t->strides();
        const size_t d = sizes.size();
        if (d == 0 || t->numel() == 0 || sizes[d - 1] > INT32_MAX)
            return false;
        cols = (int)sizes[d - 1];
        rows = t->numel() / cols;
        ld = cols;
        if (d == 2 && rows > 1) {
            ld = strides[0];
            if ((strides[1] != 1 && cols != 1) || ld < cols)
                return false;
        } else if (!t->is_contiguous()) {
            return false;
        }
        type = type_code(t->scalar_type());
        p = t->data_ptr();
        return type >= 0 && rows <= INT32_MAX;
    }
};

// A float32 vector of n values; None where `maybe`.
bool vector_of(PyObject *o, int64_t n, bool maybe, float *&p)
{
    p = nullptr;
    if (o == Py_None)
        return maybe;
    const at::Tensor *t;
    if (!tensor_of(o, t) || t->scalar_type() != at::kFloat || t->dim() != 1 || t->numel() != n || !t->is_contiguous())
        return false;
    p = static_cast<float *>(t->data_ptr());
    return true;
}

at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like)
{
    return at::Tensor(at::detail::empty_cuda(sizes, type, like.device(), std::nullopt));
}

hipStream_t stream_of(const at::Tensor &t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

// The tensors as a tuple, or None if the call was refused.
template <typename... T>
PyObject *result(int rc, const T &...t)
{
    if (rc != CONVIMG_OK)
        Py_RETURN_NONE;
    constexpr int n = sizeof...(T);
    PyObject *items[n] = {THPVariable_Wrap(t)...};
    for (PyObject *o : items)
        if (!o) {
            for (PyObject *q : items)
                Py_XDECREF(q);
            return nullptr;
        }
    if (n == 1)
        return items[0];
    PyObject *tuple = PyTuple_New(n);
    for (int i = 0; i < n; ++i) {
        if (tuple)
            PyTuple_SET_ITEM(tuple, i, items[i]);
        else
            Py_DECREF(items[i]);
    }
    return tuple;
}

// Packed rows as (codes, scales, rows, columns).
PyObject *packed_result(int rc, const at::Tensor &codes, const at::Tensor &scales, int64_t rows, int64_t cols)
{
    if (rc != CONVIMG_OK)
        Py_RETURN_NONE;
    return Py_BuildValue("(NNLL)", THPVariable_Wrap(codes), THPVariable_Wrap(scales), (long long)rows, (long long)cols);
}

// Calls the C ABI without the interpreter's lock.
template <typename F>
int unlocked(F &&f)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return rc;
}

// Packed rows to write.
struct Packed {
    at::Tensor codes, scales;
    int64_t rows, cols;

    Packed(int64_t r, int64_t c, const at::Tensor &like) : rows(r), cols(c)
    {
        const int64_t nb = (c + 31) / 32;
        codes = fresh({r, nb * 16}, at::kByte, like);
        scales = fresh({(nb + 3) / 4, r, 4}, at::kByte, like);
    }
};

// Packed rows to read.
struct Given {
    const at::Tensor *codes = nullptr, *scales = nullptr;
    int rows = 0, cols = 0;

    // (codes, scales, rows, columns)
    bool of(PyObject *o)
    {
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4)
            return false;
        const long r = PyLong_AsLong(PyTuple_GET_ITEM(o, 2)), c = PyLong_AsLong(PyTuple_GET_ITEM(o, 3));
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return false;
        }
        if (r <= 0 || c <= 0 || r > INT32_MAX || c > INT32_MAX || !tensor_of(PyTuple_GET_ITEM(o, 0), codes)
            || !tensor_of(PyTuple_GET_ITEM(o, 1), scales))
            return false;
        rows = (int)r;
        cols = (int)c;
        const int64_t nb = (c + 31) / 32;
        return codes->scalar_type() == at::kByte && scales->scalar_type() == at::kByte
            && codes->sizes() == at::IntArrayRef({r, nb * 16}) && scales->sizes() == at::IntArrayRef({(nb + 3) / 4, r, 4})
            && codes->is_contiguous() && scales->is_contiguous();
    }
};

// Runs f; a C++ exception (an allocation that fails) becomes torch's Python
// exception for it.
template <typename F>
PyObject *guarded(F &&f)
{
    HANDLE_TH_ERRORS
    return f();
    END_HANDLE_TH_ERRORS
}

#define ARGS(n)                                                                                                        \
    if (count != (n)) {                                                                                                \
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");                                                 \
        return nullptr;                                                                                                \
    }

// (x, gamma, beta, eps, out_dtype, stats)
PyObject *layer_norm(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    ARGS(6)
    return guarded([&]() -> PyObject * {
        Rows x;
        float *g, *b;
        at::ScalarType t;
        if (!x.of(a[0]) || !vector_of(a[1], x.cols, true, g) || !vector_of(a[2], x.cols, true, b)
            || !PyFloat_Check(a[3]) || !type_of(a[4], x.t->scalar_type(), t) || !PyBool_Check(a[5]))
            Py_RETURN_NONE;
        const float eps = (float)PyFloat_AS_DOUBLE(a[3]);
        const auto sizes = x.t->sizes();
        const at::Tensor y = fresh(sizes, t, *x.t);
        const hipStream_t s = stream_of(*x.t);
        if (a[5] != Py_True) {
            return result(unlocked([&] {
                              return p_layer_norm_fwd(x.p, x.ld, g, b, x.rows, x.cols, eps, x.type, type_code(t),
                                                      y.data_ptr(), nullptr, nullptr, s);
                          }),
                          y);
        }
        const at::Tensor mean = fresh(sizes.slice(0, sizes.size() - 1), at::kFloat, *x.t),
                         rstd = fresh(sizes.slice(0, sizes.size() - 1), at::kFloat, *x.t);
        return result(unlocked([&] {
                          return p_layer_norm_fwd(x.p, x.ld, g, b, x.rows, x.cols, eps, x.type, type_code(t),
                                                  y.data_ptr(), mean.data_ptr<float>(), rstd.data_ptr<float>(), s);
                      }),
                      y, mean, rstd);
    });
}

// (x, gamma, beta, eps): packed rows
PyObject *layer_norm_mxfp4(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    ARGS(4)
    return guarded([&]() -> PyObject * {
        Rows x;
        float *g, *b;
        if (!x.of(a[0]) || !vector_of(a[1], x.cols, true, g) || !vector_of(a[2], x.cols, true, b)
            || !PyFloat_Check(a[3]))
            Py_RETURN_NONE;
        const float eps = (float)PyFloat_AS_DOUBLE(a[3]);
        const Packed q(x.rows, x.cols, *x.t);
        const hipStream_t s = stream_of(*x.t);
        const int rc = unlocked([&] {
            return p_layer_norm_fwd_mxfp4(x.p, x.ld, g, b, x.rows, x.cols, eps, x.type, q.codes.data_ptr(),
                                          q.scales.data_ptr(), nullptr, nullptr, s);
        });
        return packed_result(rc, q.codes, q.scales, q.rows, q.cols);
    });
}

// (dy, x, gamma, mean, rstd, dx_dtype)
PyObject *layer_norm_bwd_call(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    ARGS(6)
    return guarded([&]() -> PyObject * {
        Rows dy, x;
        float *g;
        const at::Tensor *mean, *rstd;
        at::ScalarType t;
        if (!dy.of(a[0]) || !x.of(a[1]) || dy.t->sizes() != x.t->sizes() || !vector_of(a[2], x.cols, true, g)
            || !tensor_of(a[3], mean) || !tensor_of(a[4], rstd) || mean->scalar_type() != at::kFloat
            || rstd->scalar_type() != at::kFloat || mean->numel() != x.rows || rstd->numel() != x.rows
            || !mean->is_contiguous() || !rstd->is_contiguous() || !type_of(a[5], x.t->scalar_type(), t))
            Py_RETURN_NONE;
        size_t need = 0;
        if (p_layer_norm_bwd_workspace(x.rows, x.cols, &need) != CONVIMG_OK)
            Py_RETURN_NONE;
        const at::Tensor dx = fresh(x.t->sizes(), t, *x.t), dgamma = fresh({x.cols}, at::kFloat, *x.t),
                         dbeta = fresh({x.cols}, at::kFloat, *x.t), ws = fresh({(int64_t)need}, at::kByte, *x.t);
        const hipStream_t s = stream_of(*x.t);
        return result(unlocked([&] {
                          return p_layer_norm_bwd(dy.p, dy.ld, x.p, x.ld, g, mean->data_ptr<float>(),
                                                  rstd->data_ptr<float>(), x.rows, x.cols, dy.type, x.type,
                                                  type_code(t), dx.data_ptr(), dgamma.data_ptr<float>(),
                                                  dbeta.data_ptr<float>(), ws.data_ptr(), need, s);
                      }),
                      dx, dgamma, dbeta);
    });
}

// (x, transpose): packed rows
PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    ARGS(2)
    return guarded([&]() -> PyObject * {
        Rows x;
        if (!x.of(a[0]) || !PyBool_Check(a[1]))
            Py_RETURN_NONE;
        const bool tr = a[1] == Py_True;
        const Packed q(tr ? x.cols : x.rows, tr ? x.rows : x.cols, *x.t);
        const hipStream_t s = stream_of(*x.t);
        const int rc = unlocked([&] {
            return p_mxfp4_quantize(x.p, x.ld, (int)x.rows, x.cols, x.type, tr, q.codes.data_ptr(),
                                    q.scales.data_ptr(), s);
        });
        return packed_result(rc, q.codes, q.scales, q.rows, q.cols);
    });
}

// (q, dtype)
PyObject *dequantize(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    ARGS(2)
    return guarded([&]() -> PyObject * {
        Given q;
        at::ScalarType t;
        if (!q.of(a[0]) || a[1] == Py_None || !type_of(a[1], at::kFloat, t))
            Py_RETURN_NONE;
        const at::Tensor out = fresh({q.rows, q.cols}, t, *q.codes);
        const hipStream_t s = stream_of(out);
        return result(unlocked([&] {
                          return p_mxfp4_dequantize(q.codes->data_ptr(), q.scales->data_ptr(), q.rows, q.cols,
                                                    type_code(t), out.data_ptr(), s);
                      }),
                      out);
    });
}

// (x, w, bias, out_dtype)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    ARGS(4)
    return guarded([&]() -> PyObject * {
        Given w, q;
        Rows x;
        float *b;
        at::ScalarType t;
        if (!w.of(a[1]) || !vector_of(a[2], w.rows, true, b))
            Py_RETURN_NONE;
        const bool packed = PyTuple_Check(a[0]);
        if (packed ? !q.of(a[0]) || q.cols != w.cols || !type_of(a[3], at::kBFloat16, t)
                   : !x.of(a[0]) || x.cols != w.cols || !type_of(a[3], x.t->scalar_type(), t))
            Py_RETURN_NONE;
        const int M = packed ? q.rows : (int)x.rows, type = packed ? CONVIMG_MXFP4 : x.type;
        size_t need = 0;
        if (p_mxfp4_linear_workspace(M, w.rows, w.cols, type, &need) != CONVIMG_OK)
            Py_RETURN_NONE;
        c10::SmallVector<int64_t, 8> sizes;
        if (packed)
            sizes.push_back(M);
        else
            sizes.append(x.t->sizes().begin(), x.t->sizes().end() - 1);
        sizes.push_back(w.rows);
        const at::Tensor out = fresh(sizes, t, *w.codes);
        at::Tensor ws;
        if (need)
            ws = fresh({(int64_t)need}, at::kByte, out);
        const hipStream_t s = stream_of(out);
        return result(unlocked([&] {
                          return p_mxfp4_linear_fwd(packed ? q.codes->data_ptr() : x.p, packed ? w.cols : x.ld,
                                                    packed ? q.scales->data_ptr() : nullptr, type,
                                                    w.codes->data_ptr(), w.scales->data_ptr(), b, M, w.rows, w.cols,
                                                    type_code(t), out.data_ptr(), need ? ws.data_ptr() : nullptr,
                                                    need, s);
                      }),
                      out);
    });
}

// (dy, x, w, dx_dtype)
PyObject *linear_bwd(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    ARGS(4)
    return guarded([&]() -> PyObject * {
        Rows dy, x, w;
        at::ScalarType t;
        if (!dy.of(a[0]) || !x.of(a[1]) || !w.of(a[2]) || w.t->dim() != 2 || w.rows != dy.cols || w.cols != x.cols
            || dy.t->dim() != x.t->dim()
            || dy.t->sizes().slice(0, dy.t->dim() - 1) != x.t->sizes().slice(0, x.t->dim() - 1) || w.type != x.type
            || !type_of(a[3], x.t->scalar_type(), t))
            Py_RETURN_NONE;
        const int M = (int)x.rows, N = dy.cols, K = x.cols;
        size_t need = 0;
        if (p_mxfp4_linear_bwd_workspace(M, N, K, &need) != CONVIMG_OK)
            Py_RETURN_NONE;
        const at::Tensor dx = fresh(x.t->sizes(), t, *x.t), dw = fresh({N, K}, at::kFloat, *x.t),
                         db = fresh({N}, at::kFloat, *x.t), ws = fresh({(int64_t)need}, at::kByte, *x.t);
        const hipStream_t s = stream_of(*x.t);
        return result(unlocked([&] {
                          return p_mxfp4_linear_bwd(dy.p, dy.ld, dy.type, x.p, x.ld, w.p, w.ld, x.type, M, N, K,
                                                    type_code(t), dx.data_ptr(), dw.data_ptr<float>(),
                                                    db.data_ptr<float>(), ws.data_ptr(), need, s);
                      }),
                      dx, dw, db);
    });
}

// bind(name, address): a C entry point.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    ARGS(2)
    const char *name = PyUnicode_AsUTF8(a[0]);
    void *p = PyLong_AsVoidPtr(a[1]);
    if (!name || PyErr_Occurred())
        return nullptr;
#define BIND(f)                                                                                                        \
    if (!strcmp(name, #f)) {                                                                                           \
        p_##f = reinterpret_cast<decltype(p_##f)>(p);                                                                  \
        Py_RETURN_NONE;                                                                                                \
    }
    BIND(layer_norm_fwd)
    BIND(layer_norm_fwd_mxfp4)
    BIND(layer_norm_bwd)
    BIND(layer_norm_bwd_workspace)
    BIND(mxfp4_quantize)
    BIND(mxfp4_dequantize)
    BIND(mxfp4_linear_fwd)
    BIND(mxfp4_linear_workspace)
    BIND(mxfp4_linear_bwd)
    BIND(mxfp4_linear_bwd_workspace)
    PyErr_SetString(PyExc_KeyError, name);
    return nullptr;
}

template <typename F>
PyMethodDef method(const char *name, F f)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method("bind", bind),
                         method("layer_norm", layer_norm),
                         method("layer_norm_mxfp4", layer_norm_mxfp4),
                         method("layer_norm_bwd", layer_norm_bwd_call),
                         method("quantize", quantize),
                         method("dequantize", dequantize),
                         method("linear", linear),
                         method("linear_bwd", linear_bwd),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rows", "The row operators' calls in their common case.", -1, methods,
                      nullptr,               nullptr, nullptr,                                         nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rows() { return PyModule_Create(&module); }
