// binding.cpp -- the call of moe_linear from Python without the interpreter's
// part of it: a product of a few tokens takes the GPU 4 us, its arguments'
// checks, the output's allocation and the call through ctypes take the host 8.
//
// linear(x, w, bias, act, gated, residual, out, out_dtype) checks what the
// Python form checks, and returns the output, or NotImplemented where anything
// is not as the product wants it: the Python form then says what.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"

namespace {

moe_status (*g_linear)(const moe_linear_args*, moe_stream_t) = nullptr;

// A [rows, cols] matrix of the type on the device, its columns next to one
// another: its row stride, else -1.
int64_t row_stride(const at::Tensor& t, int64_t rows, int64_t cols, at::ScalarType type, int dev) {
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != 2 ||
        t.size(0) != rows || t.size(1) != cols || (t.stride(1) != 1 && cols > 1))
        return -1;
    // the stride of a single row is of no account
    return rows > 1 ? t.stride(0) : (cols + 7) / 8 * 8;
}

bool float_type(at::ScalarType t, int* code) {
    *code = t == at::kFloat ? MOE_FLOAT_F32 : MOE_FLOAT_BF16;
    return t == at::kFloat || t == at::kBFloat16;
}

// The output, or null where the Python form has to look (no error is set).
PyObject* run(PyObject* const* args) {
    if (!THPVariable_Check(args[0]) || !THPVariable_Check(args[1])) return nullptr;
    const at::Tensor& x = THPVariable_Unpack(args[0]);
    const at::Tensor& w = THPVariable_Unpack(args[1]);
    if (!x.is_cuda() || x.dim() != 2 || w.dim() != 2) return nullptr;
    const int dev = x.get_device();
    if (dev != c10::cuda::current_device()) return nullptr;
    const long act = PyLong_AsLong(args[3]);
    const int gated = PyObject_IsTrue(args[4]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return nullptr;
    }
    const int64_t M = x.size(0), K = x.size(1), rows = w.size(0);
    if (M > INT32_MAX || K > INT32_MAX || rows > INT32_MAX || (gated && rows % 2)) return nullptr;
    const int64_t N = gated ? rows / 2 : rows;

    at::ScalarType type = at::kBFloat16;
    if (args[6] != Py_None) {
        if (!THPVariable_Check(args[6])) return nullptr;
        type = THPVariable_Unpack(args[6]).scalar_type();
    }
    if (args[7] != Py_None) {
        if (!THPDtype_Check(args[7])) return nullptr;
        type = reinterpret_cast<THPDtype*>(args[7])->scalar_type;
    }
    moe_linear_args a = {};
    if (!float_type(type, &a.out_type)) return nullptr;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.act = act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH ? -1 : static_cast<int>(act);
    a.gated = gated;
    a.ldx = row_stride(x, M, K, at::kBFloat16, dev);
    a.ldw = row_stride(w, rows, K, at::kBFloat16, dev);
    if (a.ldx < 0 || a.ldw < 0) return nullptr;
    a.x = x.const_data_ptr();
    a.w = w.const_data_ptr();
    if (args[2] != Py_None) {
        if (!THPVariable_Check(args[2])) return nullptr;
        const at::Tensor& b = THPVariable_Unpack(args[2]);
        if (!b.is_cuda() || b.get_device() != dev || b.dim() != 1 || b.size(0) != rows ||
            !b.is_contiguous() || !float_type(b.scalar_type(), &a.bias_type))
            return nullptr;
        a.bias = b.const_data_ptr();
    }
    if (args[5] != Py_None) {
        if (!THPVariable_Check(args[5])) return nullptr;
        const at::Tensor& r = THPVariable_Unpack(args[5]);
        a.ldr = row_stride(r, M, N, type, dev);
        if (a.ldr < 0) return nullptr;
        a.residual = r.const_data_ptr();
    }
    at::Tensor out;
    if (args[6] != Py_None) {
        out = THPVariable_Unpack(args[6]);
        a.ldo = row_stride(out, M, N, type, dev);
        if (a.ldo < 0) return nullptr;
    } else {
        out = at::empty({M, N}, x.options().dtype(type).requires_grad(false));
        a.ldo = N;
    }
    a.out = out.mutable_data_ptr();
    if (g_linear(&a, c10::cuda::getCurrentCUDAStream(dev).stream()) != MOE_OK) return nullptr;
    if (args[6] != Py_None) {
        Py_INCREF(args[6]);
        return args[6];
    }
    return THPVariable_Wrap(std::move(out));
}

PyObject* linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 8 || !g_linear) {
        PyErr_SetString(PyExc_TypeError, "linear: eight arguments, after init");
        return nullptr;
    }
    PyObject* out = nullptr;
    try {
        out = run(args);
    } catch (const std::exception&) {      // (a tensor without memory, say)
        PyErr_Clear();
    }
    if (out || PyErr_Occurred()) return out;
    Py_RETURN_NOTIMPLEMENTED;
}

// init(address of moe_linear)
PyObject* init(PyObject*, PyObject* arg) {
    void* p = PyLong_AsVoidPtr(arg);
    if (PyErr_Occurred()) return nullptr;
    g_linear = reinterpret_cast<decltype(g_linear)>(p);
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL,
     nullptr},
    {"init", init, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
