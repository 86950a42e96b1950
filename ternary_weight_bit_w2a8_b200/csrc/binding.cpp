// binding.cpp -- the 4-bit floating point entry points for torch tensors.
//
// Argument marshalling only, as everywhere in the Python package: checks,
// output tensors, the current stream, then the C entry point of the same name.
// It is native because these calls are short: a decode step takes 2 to 10 us on
// the GPU, and the same checks written in Python with the call through ctypes
// took 6 us beside the launch.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "bitnet_b200.h"

namespace {

PyObject *g_error = nullptr;  // BitnetError

struct Refused {
    std::string what;
};
[[noreturn]] void refuse(const std::string &what) { throw Refused{what}; }

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

std::string shown(const at::Tensor &t) {
    std::string s = std::string(c10::toString(t.scalar_type())) + " [";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "] on " + t.device().str();
}

int64_t integer(PyObject *o, const char *name) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be an integer");
    }
    return v;
}

int format_of(PyObject *o) {
    const int64_t f = integer(o, "fmt");
    if (f != BITNET_FP4_MX && f != BITNET_FP4_NV) refuse("fmt must be BITNET_FP4_MX or BITNET_FP4_NV");
    return (int)f;
}

int float_type(at::ScalarType t, const char *name) {
    switch (t) {
        case at::kBFloat16: return BITNET_BF16;
        case at::kHalf: return BITNET_FP16;
        case at::kFloat: return BITNET_FP32;
        default: refuse(std::string(name) + " must be bfloat16, float16 or float32, not " + c10::toString(t));
    }
}

c10::Device device_of(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    return t.device();
}

void on_device(const at::Tensor &t, c10::Device d, const char *name) {
    if (t.device() != d) refuse(std::string(name) + " must be on the call's CUDA device, not " + t.device().str());
}

// Row stride of a 2-D tensor whose rows are contiguous.
int64_t row_stride(const at::Tensor &t, const char *name) {
    if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
        refuse(std::string(name) + " must be 2-D with contiguous rows, not " + shown(t));
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// Pointer of a float32 tensor of one value (null for None).
float *scalar(PyObject *o, c10::Device d, const char *name) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kFloat || t.device() != d || t.numel() != 1)
        refuse(std::string(name) + " must be a float32 tensor of one value on the call's CUDA device, not " + shown(t));
    return static_cast<float *>(t.data_ptr());
}

int64_t code_width(int64_t K) { return (K + 127) / 128 * 64; }
int64_t scale_bytes(int64_t rows, int64_t K, int fmt) {
    return (rows + 127) / 128 * ((K + 127) / 128) * (fmt == BITNET_FP4_MX ? 512 : 1024);
}

struct Matrix {
    uint8_t *codes, *scales;
    int64_t rows;
};
Matrix matrix(PyObject *oc, PyObject *os, int64_t K, int fmt, c10::Device d, const char *name) {
    const at::Tensor &c = tensor(oc, name);
    const at::Tensor &s = tensor(os, (std::string("the scales of ") + name).c_str());
    if (K < 0) refuse("K must not be negative");
    if (c.dim() != 2 || c.size(1) != code_width(K) || c.scalar_type() != at::kByte || c.device() != d || !c.is_contiguous())
        refuse(std::string(name) + " must be a contiguous uint8 tensor [rows, " + std::to_string(code_width(K)) + "] for K = " +
               std::to_string(K) + " on the call's CUDA device, not " + shown(c));
    const int64_t need = scale_bytes(c.size(0), K, fmt);
    if (s.scalar_type() != at::kByte || s.device() != d || !s.is_contiguous() || s.numel() < need)
        refuse(std::string("the scales of ") + name + " must be a contiguous uint8 tensor of " + std::to_string(need) +
               " bytes on the call's CUDA device, not " + shown(s));
    return {static_cast<uint8_t *>(c.data_ptr()), static_cast<uint8_t *>(s.data_ptr()), c.size(0)};
}

at::Tensor fresh(at::IntArrayRef size, at::ScalarType type, c10::Device d) {
    return at::detail::empty_cuda(size, type, d, std::nullopt);
}

// y as given (of the type asked for, if one is), or a new [rows, cols] of that type (bfloat16 if none).
at::Tensor output(PyObject *oy, PyObject *odtype, int64_t rows, int64_t cols, c10::Device d, int64_t *ld) {
    at::ScalarType type = at::kBFloat16;
    if (odtype != Py_None) {
        if (!THPDtype_Check(odtype)) refuse("dtype must be a torch.dtype");
        type = reinterpret_cast<THPDtype *>(odtype)->scalar_type;
    }
    if (oy == Py_None) {
        float_type(type, "dtype");
        *ld = cols;
        return fresh({rows, cols}, type, d);
    }
    at::Tensor y = tensor(oy, "y");
    on_device(y, d, "y");
    if (odtype != Py_None && y.scalar_type() != type)
        refuse(std::string("dtype is ") + c10::toString(type) + ", y is " + shown(y));
    *ld = row_stride(y, "y");
    if (y.size(0) != rows || y.size(1) != cols)
        refuse("y must be [" + std::to_string(rows) + ", " + std::to_string(cols) + "], not " + shown(y));
    return y;
}

// The C call without the interpreter lock; its status as BitnetError.
struct CallFailed {};
template <typename F>
void call(const char *where, F f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f();
    Py_END_ALLOW_THREADS;
    if (rc == BITNET_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "is", rc, where);
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw CallFailed{};
}

// Runs f with C++ exceptions turned into Python ones.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments are needed, not %zd", want, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
    } catch (const CallFailed &) {
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *type = torch != nullptr ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type != nullptr) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

void *stream_of(c10::Device d) { return c10::cuda::getCurrentCUDAStream(d.index()).stream(); }

// (x, g)
PyObject *tensor_scale(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 2, [&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const c10::Device d = device_of(x, "x");
        const c10::cuda::CUDAGuard on(d);
        const int64_t ld = row_stride(x, "x");
        const int type = float_type(x.scalar_type(), "x");
        at::Tensor g = a[1] == Py_None ? fresh({1}, at::kFloat, d) : tensor(a[1], "g");
        float *gp = a[1] == Py_None ? static_cast<float *>(g.data_ptr()) : scalar(a[1], d, "g");
        call("bitnet_fp4_tensor_scale", [&] {
            return bitnet_fp4_tensor_scale(x.data_ptr(), type, x.size(0), x.size(1), ld, gp, stream_of(d));
        });
        return THPVariable_Wrap(std::move(g));
    });
}

// (x, fmt, g, codes, scales)
PyObject *quant(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const c10::Device d = device_of(x, "x");
        const c10::cuda::CUDAGuard on(d);
        const int fmt = format_of(a[1]);
        const int64_t ld = row_stride(x, "x"), rows = x.size(0), K = x.size(1);
        const int type = float_type(x.scalar_type(), "x");
        if ((a[3] == Py_None) != (a[4] == Py_None)) refuse("codes and scales are given together");
        at::Tensor codes, scales;
        if (a[3] == Py_None) {
            codes = fresh({rows, code_width(K)}, at::kByte, d);
            scales = fresh({scale_bytes(rows, K, fmt)}, at::kByte, d);
        } else {
            if (matrix(a[3], a[4], K, fmt, d, "codes").rows != rows) refuse("codes and x differ in their rows");
            codes = tensor(a[3], "codes");
            scales = tensor(a[4], "scales");
        }
        const float *g = scalar(a[2], d, "g");
        call("bitnet_fp4_quant", [&] {
            return bitnet_fp4_quant(x.data_ptr(), type, rows, K, ld, fmt, g, static_cast<uint8_t *>(codes.data_ptr()),
                                    static_cast<uint8_t *>(scales.data_ptr()), stream_of(d));
        });
        PyObject *pc = THPVariable_Wrap(std::move(codes)), *ps = THPVariable_Wrap(std::move(scales));
        PyObject *r = pc != nullptr && ps != nullptr ? PyTuple_Pack(2, pc, ps) : nullptr;
        Py_XDECREF(pc);
        Py_XDECREF(ps);
        return r;
    });
}

// (codes, scales, K, fmt, g, dtype, y)
PyObject *dequant(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const c10::Device d = device_of(tensor(a[0], "codes"), "codes");
        const c10::cuda::CUDAGuard on(d);
        const int64_t K = integer(a[2], "K");
        const int fmt = format_of(a[3]);
        const Matrix m = matrix(a[0], a[1], K, fmt, d, "codes");
        int64_t ld = 0;
        at::Tensor y = output(a[6], a[5], m.rows, K, d, &ld);
        const int type = float_type(y.scalar_type(), "y");
        const float *g = scalar(a[4], d, "g");
        call("bitnet_fp4_dequant", [&] {
            return bitnet_fp4_dequant(m.codes, m.scales, m.rows, K, fmt, g, y.data_ptr(), type, ld, stream_of(d));
        });
        return THPVariable_Wrap(std::move(y));
    });
}

// (a, a_scales, w, w_scales, K, fmt, ga, gw, dtype, y)
PyObject *gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const c10::Device d = device_of(tensor(a[0], "a"), "a");
        const c10::cuda::CUDAGuard on(d);
        const int64_t K = integer(a[4], "K");
        const int fmt = format_of(a[5]);
        const Matrix A = matrix(a[0], a[1], K, fmt, d, "a"), W = matrix(a[2], a[3], K, fmt, d, "w");
        const float *ga = scalar(a[6], d, "ga"), *gw = scalar(a[7], d, "gw");
        int64_t ld = 0;
        at::Tensor y = output(a[9], a[8], A.rows, W.rows, d, &ld);
        const int type = float_type(y.scalar_type(), "y");
        call("bitnet_fp4_gemm", [&] {
            return bitnet_fp4_gemm(A.codes, A.scales, ga, W.codes, W.scales, gw, fmt, y.data_ptr(), type, A.rows, W.rows, K,
                                   ld, stream_of(d));
        });
        return THPVariable_Wrap(std::move(y));
    });
}

// (x, w, w_scales, fmt, ga, gw, dtype, y, ws)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const c10::Device d = device_of(x, "x");
        const c10::cuda::CUDAGuard on(d);
        const int fmt = format_of(a[3]);
        const int64_t ldx = row_stride(x, "x"), M = x.size(0), K = x.size(1);
        const int xtype = float_type(x.scalar_type(), "x");
        const Matrix W = matrix(a[1], a[2], K, fmt, d, "w");
        const float *ga = scalar(a[4], d, "ga"), *gw = scalar(a[5], d, "gw");
        int64_t ld = 0;
        at::Tensor y = output(a[7], a[6], M, W.rows, d, &ld), ws;
        const int type = float_type(y.scalar_type(), "y");
        if (a[8] != Py_None) {
            ws = tensor(a[8], "ws");
            if (ws.scalar_type() != at::kByte || ws.device() != d || !ws.is_contiguous())
                refuse("ws must be a contiguous uint8 tensor on the call's CUDA device, not " + shown(ws));
        } else {
            const int64_t need = bitnet_fp4_workspace_bytes(M, W.rows, K, fmt);
            if (need > 0) ws = fresh({need}, at::kByte, d);
        }
        void *wp = ws.defined() ? ws.data_ptr() : nullptr;
        const int64_t wb = ws.defined() ? ws.numel() : 0;
        call("bitnet_fp4_linear", [&] {
            return bitnet_fp4_linear(x.data_ptr(), xtype, ldx, ga, W.codes, W.scales, gw, fmt, y.data_ptr(), type, M, W.rows,
                                     K, ld, wp, wb, stream_of(d));
        });
        return THPVariable_Wrap(std::move(y));
    });
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(tensor_scale), FAST(quant), FAST(dequant), FAST(gemm), FAST(linear),
                           {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// Refuses a torch other than the one it was built for: their classes may differ
// where their symbols do not.
PyMODINIT_FUNC PyInit__binding(void) {
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *version = torch != nullptr ? PyObject_GetAttrString(torch, "__version__") : nullptr;
    const char *is = version != nullptr ? PyUnicode_AsUTF8(version) : nullptr;
    const bool fits = is != nullptr && std::string(is) == BINDING_TORCH;
    if (is != nullptr && !fits)
        PyErr_Format(PyExc_ImportError,
                     "the binding was built for torch " BINDING_TORCH ", this is %s: build it again with "
                     "`python -m ternary_weight_bit_w2a8_b200.build`",
                     is);
    Py_XDECREF(version);
    Py_XDECREF(torch);
    return fits ? PyModule_Create(&g_module) : nullptr;
}
