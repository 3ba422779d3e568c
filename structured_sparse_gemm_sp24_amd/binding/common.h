// What the native binding modules share: checks of tensors, outputs from torch's allocator, and calls of the C entry points
// on the current stream. Each module includes it once.
#pragma once
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>

#include "../../include/sp24.h"

namespace {

using at::Tensor;

PyObject* g_check = nullptr;       // (name, status) -> raises for a status that is not ok
PyObject* g_raw_stream = nullptr;  // device index -> handle of its current stream

constexpr auto kCodes = at::kFloat8_e4m3fn, kScales = at::kFloat8_e8m0fnu;

int64_t blocks(int64_t n) { return (n + 127) / 128; }

bool is_none(PyObject* o) { return o == nullptr || o == Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// A row-major matrix of the given type, on the first operand's device; returns its row pitch in elements (of a single
// row, which has none, its length rounded up to what every entry point takes).
int64_t matrix(const Tensor& t, const char* name, const Tensor& first, at::ScalarType type, int64_t rows, int64_t cols) {
    TORCH_CHECK_VALUE(t.device() == first.device(), name, " must be on the first operand's device");
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be of type ", type, ", not ", t.scalar_type());
    TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == rows && t.size(1) == cols, name, " must have shape (", rows, ", ", cols, "), not ", t.sizes());
    TORCH_CHECK_VALUE(cols <= 1 || t.stride(1) == 1, name, " must have unit stride along its last dimension");
    return rows > 1 ? t.stride(0) : (cols + 15) / 16 * 16;
}

void* vector(const Tensor& t, const char* name, const Tensor& first, at::ScalarType type, int64_t n) {
    TORCH_CHECK_VALUE(t.device() == first.device(), name, " must be on the first operand's device");
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be of type ", type, ", not ", t.scalar_type());
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == n && (n <= 1 || t.stride(0) == 1), name, " must be a contiguous vector of ", n, " values");
    return t.data_ptr();
}

Tensor empty(std::array<int64_t, 2> shape, at::ScalarType type, const Tensor& first) {
    const std::array<int64_t, 2> stride{shape[1], 1};
    return Tensor(at::detail::empty_strided_cuda(shape, stride, type, first.device()));
}
Tensor empty(int64_t n, at::ScalarType type, const Tensor& first) {
    const std::array<int64_t, 1> shape{n}, stride{1};
    return Tensor(at::detail::empty_strided_cuda(shape, stride, type, first.device()));
}

struct Matrix {
    Tensor t;
    int64_t ld;
    uint8_t* bytes() const { return static_cast<uint8_t*>(t.data_ptr()); }
};

// An output matrix: the one given, or a new one.
Matrix output(PyObject* o, const char* name, const Tensor& first, at::ScalarType type, int64_t rows, int64_t cols) {
    if (is_none(o)) return {empty({rows, cols}, type, first), cols};
    const Tensor& t = tensor(o, name);
    return {t, matrix(t, name, first, type, rows, cols)};
}

// The operand that the others are checked against, a matrix on a GPU.
int64_t leading(const Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.is_cuda(), "sp24 operates on device tensors only");
    TORCH_CHECK_VALUE(t.dim() == 2, name, " must be a matrix, not of shape ", t.sizes());
    return matrix(t, name, t, t.scalar_type(), t.size(0), t.size(1));
}

int float_type(const Tensor& t, const char* name) {
    switch (t.scalar_type()) {
    case at::kBFloat16: return SP24_BF16;
    case at::kHalf: return SP24_FP16;
    case at::kFloat: return SP24_FP32;
    default: break;
    }
    TORCH_CHECK_VALUE(false, name, " must be bfloat16, float16 or float32, not ", t.scalar_type());
}

int out_type(const Tensor& t) {
    return t.scalar_type() == at::kBFloat16 ? SP24_BF16 : t.scalar_type() == at::kHalf ? SP24_FP16 : t.scalar_type() == at::kFloat ? SP24_FP32 : -1;
}

void* stream_of(const Tensor& t) {
    PyObject* index = PyLong_FromLong(t.get_device());
    PyObject* handle = index ? PyObject_CallOneArg(g_raw_stream, index) : nullptr;
    Py_XDECREF(index);
    if (!handle) throw python_error();
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    return p;
}

// Calls an entry point without the interpreter's lock (a launch waits where the stream's queue is full) and raises its status.
template <typename F, typename... A>
void call(const char* name, F* entry, A... args) {
    PyThreadState* const state = PyEval_SaveThread();
    const int status = entry(args...);
    PyEval_RestoreThread(state);
    if (status == SP24_OK) return;
    Py_XDECREF(PyObject_CallFunction(g_check, "si", name, status));
    throw python_error();
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

at::ScalarType scalar_type(PyObject* dtype) {
    TORCH_CHECK_TYPE(THPDtype_Check(dtype), "out_dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(dtype)->scalar_type;
}

#define SP24_ARGS(n) TORCH_CHECK_TYPE(nargs == (n), "wrong number of arguments")

// init(check, raw_stream)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    if (nargs != 2) {
        PyErr_SetString(PyExc_TypeError, "init takes two callables");
        return nullptr;
    }
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    Py_XSETREF(g_check, a[0]);
    Py_XSETREF(g_raw_stream, a[1]);
    Py_RETURN_NONE;
}

#define SP24_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}

}  // namespace
