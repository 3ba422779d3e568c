// Native marshalling of the 8-bit operators' calls for Python: checks of the tensors, outputs and workspaces from
// torch's allocator, and the C entry points of include/sp24_fp8.h on the current stream.
//
// At one token the device work of these calls is 2.7 to 4.7 us, and the host's share decides how fast they follow one
// another: the same steps in Python over ctypes took (a call, outputs allocated) quantisation 7.1 us, norm 9.8, product
// 8.3, norm's gradients 12.5; here they take 4.4, 5.5, 3.8 and 7.5, of which a kernel launch is about 2.5.
#include "common.h"

#include "../../include/sp24_fp8.h"

namespace {

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

PyMethodDef methods[] = {SP24_METHOD(init), SP24_METHOD(quant), SP24_METHOD(rmsnorm), SP24_METHOD(rmsnorm_backward),
                         SP24_METHOD(gemm), SP24_METHOD(grad_weight), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8_binding(void) { return PyModule_Create(&module); }
