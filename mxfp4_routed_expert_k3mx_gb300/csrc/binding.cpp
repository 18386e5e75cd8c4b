// binding.cpp - the calls of k3mx_mx.h and k3mx_block.h from Python: whether the tensors are
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

#include "k3mx_block.h"

namespace {

constexpr long kUnexpected = -1;

struct {
    decltype(&k3mx_mx_quantize) quantize;
    decltype(&k3mx_mx_dequantize) dequantize;
    decltype(&k3mx_rmsnorm_mx) rmsnorm;
    decltype(&k3mx_mx_linear) linear;
    decltype(&k3mx_mx_grouped) grouped;
    decltype(&k3mx_sort) sort;
    decltype(&k3mx_dispatch) dispatch;
    decltype(&k3mx_combine) combine;
    decltype(&k3mx_combine_backward) combine_backward;
    decltype(&k3mx_situ_mx) situ;
    decltype(&k3mx_situ_mx_backward) situ_backward;
    decltype(&k3mx_rmsnorm_mx_backward) rmsnorm_backward;
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
Matrix matrix(PyObject *o, bool blocks = true, bool codes = false) {
    const at::Tensor &t = cuda_tensor(o);
    const at::ScalarType type = t.scalar_type();
    if (t.dim() != 2 || (type != at::kFloat && type != at::kBFloat16 && !(codes && type == at::kByte))) throw Unexpected();
    const int dtype = type == at::kFloat ? K3MX_F32 : type == at::kBFloat16 ? K3MX_BF16 : K3MX_E4M3;
    Matrix m{nullptr, count(t.size(0)), count(t.size(1)), dtype, t.size(1), type};
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
double real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Unexpected();
    return v;
}
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
        const double eps = real(a[6]);
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

// ----------------------------------------------------- k3mx_block.h --

template <typename T> T *optional(PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
    return o == Py_None ? nullptr : static_cast<T *>(array(o, type, shape));
}
// [tokens, topk] of int32
struct Pairs {
    int32_t *data;
    int tokens, topk;
};
Pairs pairs(PyObject *o) {
    const at::Tensor &t = cuda_tensor(o);
    if (t.dim() != 2 || t.scalar_type() != at::kInt || !t.is_contiguous()) throw Unexpected();
    return {static_cast<int32_t *>(t.data_ptr()), count(t.size(0)), count(t.size(1))};
}
struct Workspace {
    void *data;
    size_t bytes;
};
Workspace workspace(PyObject *o) {
    if (o == Py_None) return {nullptr, 0};
    const at::Tensor &t = cuda_tensor(o);
    if (!t.is_contiguous()) throw Unexpected();
    return {t.data_ptr(), t.nbytes()};
}

PyObject *sort(PyObject *, PyObject *const *a, Py_ssize_t n) {        // offsets, perm, place, idx, workspace, stream
    return guarded(n, 6, [&] {
        const Pairs p = pairs(a[3]);
        const at::Tensor &o = cuda_tensor(a[0]);
        if (o.dim() != 1) throw Unexpected();
        const int experts = count(o.size(0) - 1);
        int32_t *offsets = static_cast<int32_t *>(array(a[0], at::kInt, {experts + 1}));
        int32_t *perm = nullptr;
        if (a[1] != Py_None) {
            const at::Tensor &t = cuda_tensor(a[1]);
            if (t.numel() != (int64_t)p.tokens * p.topk) throw Unexpected();
            perm = static_cast<int32_t *>(array(a[1], at::kInt, t.sizes()));
        }
        int32_t *place = static_cast<int32_t *>(array(a[2], at::kInt, {p.tokens, p.topk}));
        const Workspace ws = workspace(a[4]);
        const k3mx_stream_t st = stream(a[5]);
        return [=] { return lib.sort(offsets, perm, place, p.data, p.tokens, p.topk, experts, ws.data, ws.bytes, st); };
    });
}

PyObject *dispatch(PyObject *, PyObject *const *a, Py_ssize_t n) {    // rows, x, place, scales, x_scales, stream
    return guarded(n, 6, [&] {
        const Matrix rows = matrix(a[0], false, true), x = matrix(a[1], false, true);
        const Pairs p = pairs(a[2]);
        if (rows.ld != rows.cols || rows.type != x.type || rows.cols != x.cols || p.tokens != x.rows) throw Unexpected();
        const bool codes = x.dtype == K3MX_E4M3;
        if ((a[3] != Py_None) != codes || (a[4] != Py_None) != codes || (codes && x.cols % 32 != 0)) throw Unexpected();
        uint8_t *scales = optional<uint8_t>(a[3], at::kByte, {rows.rows, rows.cols / 32});
        const uint8_t *xs = optional<uint8_t>(a[4], at::kByte, {x.rows, x.cols / 32});
        const k3mx_stream_t st = stream(a[5]);
        return [=] {
            return lib.dispatch(rows.data, scales, x.data, xs, x.ld, x.dtype, p.data, p.tokens, p.topk, rows.rows, x.cols, st);
        };
    });
}

PyObject *combine(PyObject *, PyObject *const *a, Py_ssize_t n) {     // y, rows, place, w, base, stream
    return guarded(n, 6, [&] {
        const Matrix y = whole(a[0], false), rows = whole(a[1], false);
        const Pairs p = pairs(a[2]);
        if (y.cols != rows.cols || p.tokens != y.rows) throw Unexpected();
        const float *w = optional<float>(a[3], at::kFloat, {p.tokens, p.topk});
        const void *base = optional<void>(a[4], y.type, {y.rows, y.cols});
        const k3mx_stream_t st = stream(a[5]);
        return [=] {
            return lib.combine(y.data, y.dtype, rows.data, rows.dtype, p.data, w, base, p.tokens, p.topk, rows.rows, y.cols, st);
        };
    });
}

PyObject *combine_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {    // drows, dw, dy, rows, place, w, stream
    return guarded(n, 7, [&] {
        const Matrix dy = matrix(a[2], false), rows = whole(a[3], false);
        const Pairs p = pairs(a[4]);
        if (dy.cols != rows.cols || p.tokens != dy.rows) throw Unexpected();
        void *drows = array(a[0], rows.type, {rows.rows, rows.cols});
        float *dw = static_cast<float *>(array(a[1], at::kFloat, {p.tokens, p.topk}));
        const float *w = static_cast<const float *>(array(a[5], at::kFloat, {p.tokens, p.topk}));
        const k3mx_stream_t st = stream(a[6]);
        return [=] {
            return lib.combine_backward(drows, dw, dy.data, dy.ld, dy.dtype, rows.data, rows.dtype, p.data, w, p.tokens, p.topk,
                                        rows.rows, rows.cols, st);
        };
    });
}

PyObject *situ_mx(PyObject *, PyObject *const *a, Py_ssize_t n) {     // codes, scales, gu, saved, saved_scales, stream
    return guarded(n, 6, [&] {
        const Matrix gu = matrix(a[2]);
        if (gu.cols % 64 != 0 || (a[3] == Py_None) != (a[4] == Py_None)) throw Unexpected();
        const int inter = gu.cols / 2;
        uint8_t *codes = bytes(a[0], {gu.rows, inter}), *scales = bytes(a[1], {gu.rows, inter / 32});
        uint8_t *saved = optional<uint8_t>(a[3], at::kByte, {gu.rows, gu.cols});
        uint8_t *ss = optional<uint8_t>(a[4], at::kByte, {gu.rows, gu.cols / 32});
        const k3mx_stream_t st = stream(a[5]);
        return [=] { return lib.situ(codes, scales, saved, ss, gu.data, gu.ld, gu.dtype, gu.rows, inter, st); };
    });
}

PyObject *situ_mx_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {    // dgu, dh, saved, saved_scales, stream
    return guarded(n, 5, [&] {
        const Matrix dh = matrix(a[1]);
        if (dh.cols > INT32_MAX / 2) throw Unexpected();
        void *dgu = array(a[0], dh.type, {dh.rows, 2 * dh.cols});
        const uint8_t *saved = bytes(a[2], {dh.rows, 2 * dh.cols}), *ss = bytes(a[3], {dh.rows, dh.cols / 16});
        const k3mx_stream_t st = stream(a[4]);
        return [=] { return lib.situ_backward(dgu, dh.data, dh.ld, dh.dtype, saved, ss, dh.rows, dh.cols, st); };
    });
}

// dx, dweight, dn, saved, saved_scales, weight, eps, workspace, dres, stream
PyObject *rmsnorm_mx_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const Matrix dn = matrix(a[2]);
        void *dx = array(a[0], dn.type, {dn.rows, dn.cols});
        float *dweight = static_cast<float *>(array(a[1], at::kFloat, {dn.cols}));
        const uint8_t *saved = bytes(a[3], {dn.rows, dn.cols}), *ss = bytes(a[4], {dn.rows, dn.cols / 32});
        const uint16_t *g = static_cast<const uint16_t *>(array(a[5], at::kBFloat16, {dn.cols}));
        const double eps = real(a[6]);
        const Workspace ws = workspace(a[7]);
        const void *dres = optional<void>(a[8], dn.type, {dn.rows, dn.cols});
        const k3mx_stream_t st = stream(a[9]);
        return [=] {
            return lib.rmsnorm_backward(dx, dweight, dn.data, dn.ld, dres, dn.dtype, saved, ss, g, static_cast<float>(eps), dn.rows,
                                        dn.cols, ws.data, ws.bytes, st);
        };
    });
}

// `count` addresses of C functions from Python; false with an exception set
bool addresses(const char *name, PyObject *const *a, Py_ssize_t n, Py_ssize_t count, void **p) {
    if (n != count) {
        PyErr_Format(PyExc_TypeError, "%s: %zd addresses expected", name, count);
        return false;
    }
    for (Py_ssize_t i = 0; i < n; i++) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s: null address", name);
            return false;
        }
    }
    return true;
}

// bind(addresses of the five C functions of k3mx_mx.h)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[5];
    if (!addresses("bind", a, n, 5, p)) return nullptr;
    lib.quantize = reinterpret_cast<decltype(lib.quantize)>(p[0]);
    lib.dequantize = reinterpret_cast<decltype(lib.dequantize)>(p[1]);
    lib.rmsnorm = reinterpret_cast<decltype(lib.rmsnorm)>(p[2]);
    lib.linear = reinterpret_cast<decltype(lib.linear)>(p[3]);
    lib.grouped = reinterpret_cast<decltype(lib.grouped)>(p[4]);
    Py_RETURN_NONE;
}

// bind_block(addresses of the seven of k3mx_block.h)
PyObject *bind_block(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[7];
    if (!addresses("bind_block", a, n, 7, p)) return nullptr;
    lib.sort = reinterpret_cast<decltype(lib.sort)>(p[0]);
    lib.dispatch = reinterpret_cast<decltype(lib.dispatch)>(p[1]);
    lib.combine = reinterpret_cast<decltype(lib.combine)>(p[2]);
    lib.combine_backward = reinterpret_cast<decltype(lib.combine_backward)>(p[3]);
    lib.situ = reinterpret_cast<decltype(lib.situ)>(p[4]);
    lib.situ_backward = reinterpret_cast<decltype(lib.situ_backward)>(p[5]);
    lib.rmsnorm_backward = reinterpret_cast<decltype(lib.rmsnorm_backward)>(p[6]);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),       FAST(mx_quantize), FAST(mx_dequantize),    FAST(rmsnorm_mx),
                         FAST(mx_linear),  FAST(mx_grouped),  FAST(bind_block),       FAST(sort),
                         FAST(dispatch),   FAST(combine),     FAST(combine_backward), FAST(situ_mx),
                         FAST(situ_mx_backward),              FAST(rmsnorm_mx_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_k3mx_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__k3mx_binding() { return PyModule_Create(&module); }
