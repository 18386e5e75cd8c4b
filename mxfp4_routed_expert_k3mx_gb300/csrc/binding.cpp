// binding.cpp - the calls of k3mx_mx.h from Python: whether the tensors are
// as a call needs them, their pointers and sizes, the current stream, and the
// C function itself.
//
// Those calls last a few microseconds on the device for few rows, and asking
// each tensor its shape, type, device and layout from Python, and handing the
// answers to the C function through ctypes, took longer: 4.2 us of host time
// for quantising and 5.4 for a product, 2.2 and 2.4 from here (nearly all of
// it the launch).  A function here returns the C function's status, or
// kUnexpected where an argument is not as it should be; the Python function
// around it then says which.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "k3mx_mx.h"

namespace {

constexpr long kUnexpected = -1;

struct {
    decltype(&k3mx_mx_quantize) quantize;
    decltype(&k3mx_mx_dequantize) dequantize;
    decltype(&k3mx_rmsnorm_mx) rmsnorm;
    decltype(&k3mx_mx_linear) linear;
    decltype(&k3mx_mx_grouped) grouped;
} lib;

struct Unexpected {};

// the device that this thread's call runs on: the current one, whose stream it
// takes and whose memory all its tensors have to be in
thread_local int device;

// (the returned reference is borrowed: the caller's arguments hold it)
const at::Tensor &cuda_tensor(PyObject *o) {
    if (!THPVariable_Check(o)) throw Unexpected();
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device || t.layout() != at::kStrided || t.is_neg()) throw Unexpected();
    return t;
}
// contiguous, of a type and a shape; its address
void *array(PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor &t = cuda_tensor(o);
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) throw Unexpected();
    return t.data_ptr();
}
uint8_t *bytes(PyObject *o, at::IntArrayRef shape) { return static_cast<uint8_t *>(array(o, at::kByte, shape)); }

// A matrix of values of blocks of 32 columns; ld its row pitch, rows contiguous
struct Matrix {
    void *data;
    int rows, cols, dtype;
    int64_t ld;
    at::ScalarType type;
};
int count(int64_t n) {
    if (n < 1 || n > INT32_MAX) throw Unexpected();
    return static_cast<int>(n);
}
Matrix matrix(PyObject *o, bool blocks = true) {
    const at::Tensor &t = cuda_tensor(o);
    const at::ScalarType type = t.scalar_type();
    if (t.dim() != 2 || (type != at::kFloat && type != at::kBFloat16)) throw Unexpected();
    Matrix m{nullptr, count(t.size(0)), count(t.size(1)), type == at::kFloat ? K3MX_F32 : K3MX_BF16, t.size(1), type};
    if (blocks && m.cols % 32 != 0) throw Unexpected();
    if (t.stride(1) != 1 && m.cols > 1) throw Unexpected();
    if (m.rows > 1) m.ld = t.stride(0);
    if (m.ld < m.cols) throw Unexpected();
    m.data = t.data_ptr();
    return m;
}
Matrix whole(PyObject *o, bool blocks = true) {
    const Matrix m = matrix(o, blocks);
    if (m.ld != m.cols) throw Unexpected();
    return m;
}
int format(PyObject *o) {
    const long f = PyLong_AsLong(o);
    if (f != K3MX_MXFP4 && f != K3MX_MXFP8) throw Unexpected();
    return static_cast<int>(f);
}
int64_t code_bytes(int64_t cols, int fmt) { return fmt == K3MX_MXFP4 ? cols / 2 : cols; }
k3mx_stream_t stream(PyObject *o) {
    if (o == Py_None) return reinterpret_cast<k3mx_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
    void *p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw Unexpected();
    return static_cast<k3mx_stream_t>(p);
}

// `work` gives the C call, made without the interpreter's lock
template <typename F> PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F work) {
    long st = kUnexpected;
    if (n == want) {
        try {
            device = c10::cuda::current_device();
            auto call = work();
            Py_BEGIN_ALLOW_THREADS
            st = call();
            Py_END_ALLOW_THREADS
        } catch (...) {
            PyErr_Clear();
        }
    }
    return PyLong_FromLong(st);
}

PyObject *mx_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {          // codes, scales, x, fmt, stream
    return guarded(n, 5, [&] {
        const Matrix x = matrix(a[2]);
        const int fmt = format(a[3]);
        uint8_t *codes = bytes(a[0], {x.rows, code_bytes(x.cols, fmt)}), *scales = bytes(a[1], {x.rows, x.cols / 32});
        const k3mx_stream_t st = stream(a[4]);
        return [=] { return lib.quantize(codes, scales, x.data, x.dtype, x.rows, x.cols, x.ld, fmt, st); };
    });
}

PyObject *mx_dequantize(PyObject *, PyObject *const *a, Py_ssize_t n) {        // y, codes, scales, fmt, stream
    return guarded(n, 5, [&] {
        const Matrix y = whole(a[0]);
        const int fmt = format(a[3]);
        const uint8_t *codes = bytes(a[1], {y.rows, code_bytes(y.cols, fmt)}), *scales = bytes(a[2], {y.rows, y.cols / 32});
        const k3mx_stream_t st = stream(a[4]);
        return [=] { return lib.dequantize(y.data, y.dtype, codes, scales, y.rows, y.cols, fmt, st); };
    });
}

PyObject *rmsnorm_mx(PyObject *, PyObject *const *a, Py_ssize_t n) {  // codes, scales, sum, x, residual, weight, eps, normed, stream
    return guarded(n, 9, [&] {
        const Matrix x = matrix(a[3]);
        uint8_t *codes = bytes(a[0], {x.rows, x.cols}), *scales = bytes(a[1], {x.rows, x.cols / 32});
        if ((a[2] == Py_None) != (a[4] == Py_None)) throw Unexpected();
        void *sum = a[2] == Py_None ? nullptr : array(a[2], x.type, {x.rows, x.cols});
        const void *residual = a[4] == Py_None ? nullptr : array(a[4], x.type, {x.rows, x.cols});
        const uint16_t *g = static_cast<const uint16_t *>(array(a[5], at::kBFloat16, {x.cols}));
        const double eps = PyFloat_AsDouble(a[6]);
        if (eps == -1.0 && PyErr_Occurred()) throw Unexpected();
        uint16_t *normed = a[7] == Py_None ? nullptr : static_cast<uint16_t *>(array(a[7], at::kBFloat16, {x.rows, x.cols}));
        const k3mx_stream_t st = stream(a[8]);
        return [=] {
            return lib.rmsnorm(codes, scales, sum, normed, x.data, x.ld, residual, x.dtype, g, static_cast<float>(eps), x.rows,
                               x.cols, st);
        };
    });
}

PyObject *mx_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {            // y, codes, scales, packed, wscales, stream
    return guarded(n, 6, [&] {
        const Matrix y = whole(a[0], false);
        const at::Tensor &c = cuda_tensor(a[1]);
        if (c.dim() != 2) throw Unexpected();
        const int in = count(c.size(1));
        if (in % 32 != 0) throw Unexpected();
        const uint8_t *codes = bytes(a[1], {y.rows, in}), *scales = bytes(a[2], {y.rows, in / 32});
        const uint8_t *packed = bytes(a[3], {y.cols, in / 2}), *wscales = bytes(a[4], {y.cols, in / 32});
        const k3mx_stream_t st = stream(a[5]);
        return [=] { return lib.linear(y.data, y.dtype, codes, scales, packed, wscales, y.rows, in, y.cols, st); };
    });
}

PyObject *mx_grouped(PyObject *, PyObject *const *a, Py_ssize_t n) {  // y, codes, scales, packed, wscales, offsets, stream
    return guarded(n, 7, [&] {
        const Matrix y = whole(a[0], false);
        const at::Tensor &w = cuda_tensor(a[3]);
        if (w.dim() != 3) throw Unexpected();
        const int groups = count(w.size(0)), in = count(2 * w.size(2));
        if (in % 32 != 0) throw Unexpected();
        const uint8_t *codes = bytes(a[1], {y.rows, in}), *scales = bytes(a[2], {y.rows, in / 32});
        const uint8_t *packed = bytes(a[3], {groups, y.cols, in / 2}), *wscales = bytes(a[4], {groups, y.cols, in / 32});
        const int32_t *offsets = static_cast<const int32_t *>(array(a[5], at::kInt, {groups + 1}));
        const k3mx_stream_t st = stream(a[6]);
        return [=] { return lib.grouped(y.data, y.dtype, codes, scales, packed, wscales, offsets, groups, y.rows, in, y.cols, st); };
    });
}

// bind(addresses of the five C functions)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[5];
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind: five addresses expected");
        return nullptr;
    }
    for (int i = 0; i < 5; i++) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
            return nullptr;
        }
    }
    lib.quantize = reinterpret_cast<decltype(lib.quantize)>(p[0]);
    lib.dequantize = reinterpret_cast<decltype(lib.dequantize)>(p[1]);
    lib.rmsnorm = reinterpret_cast<decltype(lib.rmsnorm)>(p[2]);
    lib.linear = reinterpret_cast<decltype(lib.linear)>(p[3]);
    lib.grouped = reinterpret_cast<decltype(lib.grouped)>(p[4]);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),      FAST(mx_quantize), FAST(mx_dequantize), FAST(rmsnorm_mx),
                         FAST(mx_linear), FAST(mx_grouped),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_k3mx_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__k3mx_binding() { return PyModule_Create(&module); }
