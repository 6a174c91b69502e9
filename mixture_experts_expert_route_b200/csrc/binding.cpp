// binding.cpp -- the calls of moe_linear and moe_decode_forward from Python
// without the interpreter's part of them: a product of a few tokens takes the GPU
// 4 us, its arguments' checks, the output's allocation and the call through
// ctypes take the host 7.5 (here 3.9).
//
// linear(x, w, bias, act, gated, residual, out, out_dtype, status) and
// decode(dtype, x, logits, packed, scales, E, I, k, residual, out, ids, w, status,
// ws) check what the Python forms check, and return the output, or NotImplemented where anything
// is not as the entry point wants it: the Python form then says what.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "moe.h"

namespace {

decltype(&moe_linear) g_linear = nullptr;
decltype(&moe_decode_forward) g_decode = nullptr;
decltype(&moe_packed_weights_size) g_packed_size = nullptr;

// Allocation and launch may wait; other threads run meanwhile.
struct NoGil {
    PyThreadState* state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

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

// An optional status word on the device.
bool status_word(PyObject* o, int dev, int32_t** p) {
    *p = nullptr;
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kInt || t.numel() < 1)
        return false;
    *p = static_cast<int32_t*>(t.mutable_data_ptr());
    return true;
}

// A buffer of bytes on the device, whose numel is its size.
bool bytes_on(const at::Tensor& t, int dev) {
    return t.is_cuda() && t.get_device() == dev && t.scalar_type() == at::kByte && t.is_contiguous();
}

// The output that the caller gave, else the new one.
PyObject* result(PyObject* given, at::Tensor&& out) {
    if (given == Py_None) return THPVariable_Wrap(std::move(out));
    Py_INCREF(given);
    return given;
}

// The output, or null where the Python form has to look (no error is set).
PyObject* run_linear(PyObject* const* args) {
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
    if (!status_word(args[8], dev, &a.status)) return nullptr;
    at::Tensor out;
    if (args[6] != Py_None) {
        out = THPVariable_Unpack(args[6]);
        a.ldo = row_stride(out, M, N, type, dev);
        if (a.ldo < 0) return nullptr;
    }
    moe_status st;
    {
        NoGil free;
        if (!out.defined()) {
            out = at::empty({M, N}, x.options().dtype(type).requires_grad(false));
            a.ldo = N;
        }
        a.out = out.mutable_data_ptr();
        st = g_linear(&a, c10::cuda::getCurrentCUDAStream(dev).stream());
    }
    return st == MOE_OK ? result(args[6], std::move(out)) : nullptr;
}

// An optional contiguous tensor of the type and shape on the device.
bool whole(PyObject* o, int dev, at::ScalarType type, int64_t rows, int64_t cols, const void** p) {
    *p = nullptr;
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != 2 ||
        t.size(0) != rows || t.size(1) != cols || !t.is_contiguous())
        return false;
    *p = t.const_data_ptr();
    return true;
}

PyObject* run_decode(PyObject* const* args) {
    for (int i : {1, 3, 13})
        if (!THPVariable_Check(args[i])) return nullptr;
    const at::Tensor& x = THPVariable_Unpack(args[1]);
    const at::Tensor& packed = THPVariable_Unpack(args[3]);
    const at::Tensor& ws = THPVariable_Unpack(args[13]);
    if (!x.is_cuda() || x.dim() != 2) return nullptr;
    const int dev = x.get_device();
    if (dev != c10::cuda::current_device() || !bytes_on(packed, dev) || !bytes_on(ws, dev))
        return nullptr;
    const int64_t T = x.size(0), H = x.size(1);
    const long dtype = PyLong_AsLong(args[0]), E = PyLong_AsLong(args[5]),
               I = PyLong_AsLong(args[6]), k = PyLong_AsLong(args[7]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return nullptr;
    }
    if (T < 1 || T > 16 || H > INT32_MAX || E < 1 || E > INT32_MAX || I < 1 || I > INT32_MAX ||
        k < 1 || k > E || (dtype != MOE_BF16 && dtype != MOE_FP8_E4M3))
        return nullptr;
    moe_decode_args a = {};
    a.dtype = static_cast<moe_dtype>(dtype);
    a.T = static_cast<int>(T);
    a.k = static_cast<int>(k);
    a.E = static_cast<int>(E);
    a.H = static_cast<int>(H);
    a.I = static_cast<int>(I);
    if (static_cast<size_t>(packed.numel()) < g_packed_size(a.dtype, a.E, a.H, a.I)) return nullptr;
    const void *logits, *scales, *ids, *w;
    if (!whole(args[1], dev, at::kBFloat16, T, H, &a.x) ||
        !whole(args[2], dev, at::kFloat, T, E, &logits) ||
        !whole(args[4], dev, at::kFloat, E, 3, &scales) ||
        !whole(args[8], dev, at::kBFloat16, T, H, &a.residual) ||
        !whole(args[10], dev, at::kInt, T, k, &ids) || !whole(args[11], dev, at::kFloat, T, k, &w))
        return nullptr;
    a.logits = static_cast<const float*>(logits);
    a.packed = packed.const_data_ptr();
    a.scales = static_cast<const float*>(scales);
    a.ids = static_cast<int32_t*>(const_cast<void*>(ids));
    a.w = static_cast<float*>(const_cast<void*>(w));
    if (!status_word(args[12], dev, &a.status)) return nullptr;
    at::Tensor out;
    if (args[9] != Py_None) {
        const void* p;
        if (!whole(args[9], dev, at::kBFloat16, T, H, &p)) return nullptr;
        out = THPVariable_Unpack(args[9]);
    }
    moe_status st;
    {
        NoGil free;
        if (!out.defined()) out = at::empty({T, H}, x.options().requires_grad(false));
        a.out = out.mutable_data_ptr();
        st = g_decode(&a, ws.mutable_data_ptr(), static_cast<size_t>(ws.numel()),
                      c10::cuda::getCurrentCUDAStream(dev).stream());
    }
    return st == MOE_OK ? result(args[9], std::move(out)) : nullptr;
}

template <Py_ssize_t N, PyObject* (*RUN)(PyObject* const*)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N || !g_linear) {
        PyErr_SetString(PyExc_TypeError, "_binding: wrong number of arguments, or before init");
        return nullptr;
    }
    PyObject* out = nullptr;
    try {
        out = RUN(args);
    } catch (const std::exception&) {      // (a tensor without memory, say)
        PyErr_Clear();
    }
    if (out || PyErr_Occurred()) return out;
    Py_RETURN_NOTIMPLEMENTED;
}

// init(addresses of moe_linear, moe_decode_forward, moe_packed_weights_size)
PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
    void* p[3] = {};
    for (Py_ssize_t i = 0; i < n && i < 3; ++i) p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
    if (n != 3 || !p[0] || !p[1] || !p[2]) {
        PyErr_SetString(PyExc_TypeError, "init: three addresses");
        return nullptr;
    }
    g_linear = reinterpret_cast<decltype(g_linear)>(p[0]);
    g_decode = reinterpret_cast<decltype(g_decode)>(p[1]);
    g_packed_size = reinterpret_cast<decltype(g_packed_size)>(p[2]);
    Py_RETURN_NONE;
}

template <class F> PyCFunction method(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {
    {"linear", method(call<9, run_linear>), METH_FASTCALL, nullptr},
    {"decode", method(call<14, run_decode>), METH_FASTCALL, nullptr},
    {"init", method(init), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
    PyObject* m = PyModule_Create(&kModule);
    // tensors are read by the layouts of this torch: another one must not use it
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
