// Native marshalling of the 8-bit operators' calls for Python: checks of the tensors, outputs and workspaces from
// torch's allocator, and the C entry points of include/sp24_fp8.h on the current stream.
//
// At one token the device work of these calls is 2.7 to 4.7 us, and the host's share decides how fast they follow one
// another: the same steps in Python over ctypes took (a call, outputs allocated) quantisation 7.1 us, norm 9.8, product
// 8.3, norm's gradients 12.5; here they take 4.4, 5.5, 3.8 and 7.5, of which a kernel launch is about 2.5.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>

#include "../../include/sp24.h"
#include "../../include/sp24_fp8.h"

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

// quant(X, codes, scales) -> (codes, scales)
PyObject* quant(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    SP24_ARGS(3);
    const Tensor& X = tensor(a[0], "X");
    const int64_t ldx = leading(X, "X"), N = X.size(0), K = X.size(1);
    const int type = float_type(X, "X");
    const c10::DeviceGuard guard(X.device());
    const Matrix codes = output(a[1], "codes", X, kCodes, N, K), scales = output(a[2], "scales", X, kScales, N, blocks(K));
    call("sp24_quant_fp8", sp24_quant_fp8, X.data_ptr(), type, N, K, ldx, codes.bytes(), codes.ld, scales.bytes(), scales.ld, stream_of(X));
    return Py_BuildValue("(NN)", wrap(codes.t), wrap(scales.t));
    END_HANDLE_TH_ERRORS
}

// rmsnorm(X, gamma, eps, residual, H, codes, scales, rstd) -> (codes, scales, H, rstd)
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    SP24_ARGS(8);
    const Tensor& X = tensor(a[0], "X");
    const int64_t ldx = leading(X, "X"), N = X.size(0), K = X.size(1);
    const int type = float_type(X, "X");
    const auto st = X.scalar_type();
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) throw python_error();
    const c10::DeviceGuard guard(X.device());
    const void* gamma = vector(tensor(a[1], "gamma"), "gamma", X, st, K);
    TORCH_CHECK_VALUE(!is_none(a[3]) || is_none(a[4]), "H is only written with a residual");
    Matrix R{Tensor(), 0}, H{X, 0};
    if (!is_none(a[3])) {
        R.t = tensor(a[3], "residual");
        R.ld = matrix(R.t, "residual", X, st, N, K);
        H = output(a[4], "H", X, st, N, K);
    }
    const Matrix codes = output(a[5], "codes", X, kCodes, N, K), scales = output(a[6], "scales", X, kScales, N, blocks(K));
    const Tensor rstd = is_none(a[7]) ? empty(N, at::kFloat, X) : tensor(a[7], "rstd");
    float* const r = static_cast<float*>(vector(rstd, "rstd", X, at::kFloat, N));
    call("sp24_rmsnorm_fp8", sp24_rmsnorm_fp8, X.data_ptr(), type, N, K, ldx, R.t.defined() ? R.t.data_ptr() : nullptr, R.ld, gamma,
         static_cast<float>(eps), R.t.defined() ? H.t.data_ptr() : nullptr, H.ld, codes.bytes(), codes.ld, scales.bytes(), scales.ld, r, stream_of(X));
    return Py_BuildValue("(NNNN)", wrap(codes.t), wrap(scales.t), wrap(H.t), wrap(rstd));
    END_HANDLE_TH_ERRORS
}

// rmsnorm_backward(dY, H, rstd, gamma, dH, dX, dgamma) -> (dX, dgamma)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    SP24_ARGS(7);
    const Tensor &dY = tensor(a[0], "dY"), &H = tensor(a[1], "H");
    const int64_t ldh = leading(H, "H"), N = H.size(0), K = H.size(1);
    const int type = float_type(H, "H");
    const auto st = H.scalar_type();
    const c10::DeviceGuard guard(H.device());
    const int64_t lddy = matrix(dY, "dY", H, st, N, K);
    const float* rstd = static_cast<const float*>(vector(tensor(a[2], "rstd"), "rstd", H, at::kFloat, N));
    const void* gamma = vector(tensor(a[3], "gamma"), "gamma", H, st, K);
    Matrix dH{Tensor(), 0};
    if (!is_none(a[4])) dH = {tensor(a[4], "dH"), matrix(tensor(a[4], "dH"), "dH", H, st, N, K)};
    const Matrix dX = output(a[5], "dX", H, st, N, K);
    const Tensor dgamma = is_none(a[6]) ? empty(K, at::kFloat, H) : tensor(a[6], "dgamma");
    float* const dg = static_cast<float*>(vector(dgamma, "dgamma", H, at::kFloat, K));
    int64_t bytes = 0;
    call("sp24_rmsnorm_backward_bytes", sp24_rmsnorm_backward_bytes, N, K, &bytes);
    const Tensor work = empty(bytes, at::kByte, H);
    call("sp24_rmsnorm_backward", sp24_rmsnorm_backward, dY.data_ptr(), type, N, K, lddy, H.data_ptr(), ldh, rstd, gamma,
         dH.t.defined() ? dH.t.data_ptr() : nullptr, dH.ld, dX.t.data_ptr(), dX.ld, dg, work.data_ptr(), stream_of(H));
    return Py_BuildValue("(NN)", wrap(dX.t), wrap(dgamma));
    END_HANDLE_TH_ERRORS
}

// gemm(values, meta, w_scales, M, X, x_scales, out_dtype, out) -> out
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    SP24_ARGS(8);
    const Tensor &values = tensor(a[0], "values"), &meta = tensor(a[1], "meta"), &ws = tensor(a[2], "w_scales"), &X = tensor(a[4], "X"), &xs = tensor(a[5], "x_scales");
    const int64_t M = PyLong_AsLongLong(a[3]);
    if (M == -1 && PyErr_Occurred()) throw python_error();
    const int64_t ldx = leading(X, "X"), N = X.size(0), K = X.size(1), kb = blocks(K);
    matrix(X, "X", X, kCodes, N, K);
    const c10::DeviceGuard guard(X.device());
    const int64_t lds = matrix(xs, "x_scales", X, kScales, N, kb);
    // The scales first: their size bounds M, and with it the sizes computed from it.
    TORCH_CHECK_VALUE(M >= 0 && M < int64_t{1} << 40, "M must be a row count, not ", M);
    matrix(ws, "w_scales", X, kScales, blocks(M), kb);
    TORCH_CHECK_VALUE(ws.is_contiguous(), "w_scales must be contiguous");
    const int64_t tiles = (M + 15) / 16 * kb;
    const auto* v = static_cast<const uint8_t*>(vector(values, "values", X, kCodes, 1024 * tiles));
    const auto* m = static_cast<const uint8_t*>(vector(meta, "meta", X, at::kByte, 256 * tiles));
    const Matrix out = output(a[7], "out", X, is_none(a[7]) ? scalar_type(a[6]) : tensor(a[7], "out").scalar_type(), N, M);
    call("sp24_gemm_fp8", sp24_gemm_fp8, v, m, static_cast<const uint8_t*>(ws.data_ptr()), M, K, static_cast<const uint8_t*>(X.data_ptr()), N, ldx,
         static_cast<const uint8_t*>(xs.data_ptr()), lds, out.t.data_ptr(), out_type(out.t), out.ld, stream_of(X));
    return wrap(out.t);
    END_HANDLE_TH_ERRORS
}

// grad_weight(dY, X, x_scales, meta, out_dtype, out) -> out
PyObject* grad_weight(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    SP24_ARGS(6);
    const Tensor &dY = tensor(a[0], "dY"), &X = tensor(a[1], "X"), &xs = tensor(a[2], "x_scales");
    const int64_t ldx = leading(X, "X"), N = X.size(0), K = X.size(1), kb = blocks(K);
    matrix(X, "X", X, kCodes, N, K);
    TORCH_CHECK_VALUE(dY.dim() == 2, "dY must be a matrix, not of shape ", dY.sizes());
    const int64_t M = dY.size(1);
    const c10::DeviceGuard guard(X.device());
    const int64_t lddy = matrix(dY, "dY", X, at::kBFloat16, N, M), lds = matrix(xs, "x_scales", X, kScales, N, kb);
    const uint8_t* meta = nullptr;
    if (!is_none(a[3])) meta = static_cast<const uint8_t*>(vector(tensor(a[3], "meta"), "meta", X, at::kByte, 256 * ((M + 15) / 16 * kb)));
    const Matrix out = output(a[5], "out", X, is_none(a[5]) ? scalar_type(a[4]) : tensor(a[5], "out").scalar_type(), M, K);
    int64_t bytes = 0;
    call("sp24_grad_weight_fp8_bytes", sp24_grad_weight_fp8_bytes, M, K, N, &bytes);
    Tensor work;
    if (bytes) work = empty(bytes, at::kByte, X);
    call("sp24_grad_weight_fp8", sp24_grad_weight_fp8, dY.data_ptr(), N, M, lddy, static_cast<const uint8_t*>(X.data_ptr()), K, ldx,
         static_cast<const uint8_t*>(xs.data_ptr()), lds, meta, out.t.data_ptr(), out_type(out.t), out.ld,
         bytes ? work.data_ptr() : nullptr, stream_of(X));
    return wrap(out.t);
    END_HANDLE_TH_ERRORS
}

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
PyMethodDef methods[] = {SP24_METHOD(init), SP24_METHOD(quant), SP24_METHOD(rmsnorm), SP24_METHOD(rmsnorm_backward),
                         SP24_METHOD(gemm), SP24_METHOD(grad_weight), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8_binding(void) { return PyModule_Create(&module); }
