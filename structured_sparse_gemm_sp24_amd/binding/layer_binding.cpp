// Native marshalling of the layer operators' calls for Python (include/sp24_layer.h): the products of a decoding step are a
// few microseconds of device work, and a step of AdamW passes hundreds of tensors.
#include "common.h"

#include <torch/csrc/utils/tensor_dtypes.h>

#include <utility>
#include <vector>

#include "../../include/sp24_layer.h"

namespace {

int64_t integer(PyObject* o, const char* name) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    (void)name;
    return v;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

// preact: None or False for none, True for a new tensor, or the tensor to fill.
bool wants(PyObject* o) { return !is_none(o) && o != Py_False; }

const float* bias_of(PyObject* o, const Tensor& first, int64_t M) {
    return is_none(o) ? nullptr : static_cast<const float*>(vector(tensor(o, "bias"), "bias", first, at::kFloat, M));
}

PyObject* result(const Tensor& y, const Tensor& z) { return z.defined() ? Py_BuildValue("(NN)", wrap(y), wrap(z)) : wrap(y); }

// An operand of Y's shape: a matrix, or a batch of them.
struct Entries {
    Tensor t;
    int64_t ld = 0, stride = 0;
    void* data() const { return t.defined() ? t.data_ptr() : nullptr; }
};
Entries entries(const Tensor& t, const char* name, const Tensor& first, at::ScalarType type, at::IntArrayRef shape) {
    TORCH_CHECK_VALUE(t.device() == first.device(), name, " must be on the first operand's device");
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be of type ", type, ", not ", t.scalar_type());
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", not ", t.sizes());
    const int64_t d = t.dim(), rows = t.size(d - 2), cols = t.size(d - 1);
    TORCH_CHECK_VALUE(cols <= 1 || t.stride(d - 1) == 1, name, " must have unit stride along its last dimension");
    const int64_t ld = rows > 1 ? std::max(t.stride(d - 2), int64_t{0}) : std::max(t.stride(d - 2), (cols + 15) / 16 * 16);
    return {t, ld, d == 3 && t.size(0) > 1 ? t.stride(0) : 0};
}
Tensor empty_like_shape(at::IntArrayRef shape, at::ScalarType type, const Tensor& first) {
    std::vector<int64_t> stride(shape.size());
    int64_t n = 1;
    for (size_t i = shape.size(); i-- > 0; n *= shape[i]) stride[i] = n;
    return Tensor(at::detail::empty_strided_cuda(shape, stride, type, first.device()));
}
Entries made_or_given(PyObject* o, const char* name, const Tensor& first, at::ScalarType type, at::IntArrayRef shape) {
    const Tensor t = is_none(o) || o == Py_True ? empty_like_shape(shape, type, first) : tensor(o, name);
    return entries(t, name, first, type, shape);
}

// gemm_bf16(values, meta, M, X, bias, activation, residual, preact, token, out_dtype, out) -> out, or (out, preact)
PyObject* gemm_bf16(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    SP24_ARGS(11);
    const Tensor &values = tensor(a[0], "values"), &meta = tensor(a[1], "meta"), &X = tensor(a[3], "X");
    const int64_t M = integer(a[2], "M"), token = integer(a[8], "layout");
    TORCH_CHECK_VALUE(X.is_cuda(), "sp24 operates on device tensors only");
    TORCH_CHECK_VALUE(X.dim() == 2 || X.dim() == 3, "X must be 2-D, or 3-D for a batch");
    TORCH_CHECK_VALUE(M >= 0 && M < int64_t{1} << 40, "M must be a row count, not ", M);
    const int64_t d = X.dim(), N = X.size(d - (token ? 2 : 1)), K = X.size(d - (token ? 1 : 2)), batch = d == 3 ? X.size(0) : 1;
    const Entries x = entries(X, "X", X, at::kBFloat16, X.sizes());
    const c10::DeviceGuard guard(X.device());
    const int64_t tiles = (M + 15) / 16 * ((K + 63) / 64);
    const void* const v = vector(values, "values", X, at::kBFloat16, 512 * tiles);
    const auto* const m = static_cast<const uint8_t*>(vector(meta, "meta", X, at::kByte, 128 * tiles));
    const float* const bias = bias_of(a[4], X, M);
    std::vector<int64_t> shape;
    if (d == 3) shape.push_back(batch);
    shape.push_back(token ? N : M);
    shape.push_back(token ? M : N);
    const at::ScalarType type = is_none(a[10]) ? scalar_type(a[9]) : tensor(a[10], "out").scalar_type();
    TORCH_CHECK_VALUE(type == at::kBFloat16 || type == at::kFloat, "out must be bfloat16 or float32, not ", type);
    Entries R, Z;
    if (!is_none(a[6])) R = entries(tensor(a[6], "residual"), "residual", X, type, shape);
    const Entries Y = made_or_given(a[10], "out", X, type, shape);
    if (wants(a[7])) Z = made_or_given(a[7], "preact", X, type, shape);
    call("sp24_gemm_bf16_fused", sp24_gemm_bf16_fused, v, m, M, K, X.data_ptr(), N, x.ld, x.stride, bias, static_cast<int>(integer(a[5], "activation")),
         R.data(), R.ld, R.stride, Z.data(), Z.ld, Z.stride, Y.data(), out_type(Y.t), Y.ld, Y.stride, batch,
         static_cast<int>(token ? SP24_TOKEN_MAJOR : SP24_FEATURE_MAJOR), stream_of(X));
    return result(Y.t, Z.t);
    END_HANDLE_TH_ERRORS
}

// gemm_fp8(values, meta, w_scales, M, X, x_scales, bias, activation, residual, preact, out_dtype, out) -> out, or (out, preact)
PyObject* gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    SP24_ARGS(12);
    const Tensor &values = tensor(a[0], "values"), &meta = tensor(a[1], "meta"), &ws = tensor(a[2], "w_scales"), &X = tensor(a[4], "X"), &xs = tensor(a[5], "x_scales");
    const int64_t M = integer(a[3], "M");
    const int64_t ldx = leading(X, "X"), N = X.size(0), K = X.size(1), kb = blocks(K);
    matrix(X, "X", X, kCodes, N, K);
    const c10::DeviceGuard guard(X.device());
    const int64_t lds = matrix(xs, "x_scales", X, kScales, N, kb);
    TORCH_CHECK_VALUE(M >= 0 && M < int64_t{1} << 40, "M must be a row count, not ", M);
    matrix(ws, "w_scales", X, kScales, blocks(M), kb);
    TORCH_CHECK_VALUE(ws.is_contiguous(), "w_scales must be contiguous");
    const int64_t tiles = (M + 15) / 16 * kb;
    const auto* v = static_cast<const uint8_t*>(vector(values, "values", X, kCodes, 1024 * tiles));
    const auto* m = static_cast<const uint8_t*>(vector(meta, "meta", X, at::kByte, 256 * tiles));
    const float* const bias = bias_of(a[6], X, M);
    const at::ScalarType type = is_none(a[11]) ? scalar_type(a[10]) : tensor(a[11], "out").scalar_type();
    Matrix R{Tensor(), 0}, Z{Tensor(), 0};
    if (!is_none(a[8])) R = {tensor(a[8], "residual"), matrix(tensor(a[8], "residual"), "residual", X, type, N, M)};
    const Matrix out = output(a[11], "out", X, type, N, M);
    if (wants(a[9])) Z = output(a[9] == Py_True ? nullptr : a[9], "preact", X, type, N, M);
    call("sp24_gemm_fp8_fused", sp24_gemm_fp8_fused, v, m, static_cast<const uint8_t*>(ws.data_ptr()), M, K, static_cast<const uint8_t*>(X.data_ptr()), N,
         ldx, static_cast<const uint8_t*>(xs.data_ptr()), lds, bias, static_cast<int>(integer(a[7], "activation")),
         R.t.defined() ? R.t.data_ptr() : nullptr, R.ld, Z.t.defined() ? Z.t.data_ptr() : nullptr, Z.ld,
         out.t.data_ptr(), out_type(out.t), out.ld, stream_of(X));
    return result(out.t, Z.t);
    END_HANDLE_TH_ERRORS
}

// epilogue_backward(dY, preact, activation, dZ, dbias, want_dbias) -> (dZ, dbias)
PyObject* epilogue_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    SP24_ARGS(6);
    const Tensor& dY = tensor(a[0], "dY");
    const int64_t lddy = leading(dY, "dY"), N = dY.size(0), M = dY.size(1), act = integer(a[2], "activation");
    const int type = float_type(dY, "dY");
    const auto st = dY.scalar_type();
    const c10::DeviceGuard guard(dY.device());
    Matrix Z{Tensor(), 0}, dZ{dY, 0};
    if (!is_none(a[1])) Z = {tensor(a[1], "preact"), matrix(tensor(a[1], "preact"), "preact", dY, st, N, M)};
    TORCH_CHECK_VALUE(act == SP24_ACT_NONE ? !Z.t.defined() && is_none(a[3]) : Z.t.defined(),
                      act == SP24_ACT_NONE ? "without an activation dZ is dY: neither preact nor dZ is taken" : "an activation's gradient needs preact");
    if (act != SP24_ACT_NONE) dZ = output(a[3], "dZ", dY, st, N, M);
    const bool want = a[5] != Py_False || !is_none(a[4]);
    Tensor dbias, work;
    int64_t bytes = 0;
    if (want) {
        dbias = is_none(a[4]) ? empty(M, at::kFloat, dY) : tensor(a[4], "dbias");
        vector(dbias, "dbias", dY, at::kFloat, M);
        call("sp24_epilogue_backward_bytes", sp24_epilogue_backward_bytes, N, M, &bytes);
        if (bytes) work = empty(bytes, at::kByte, dY);
    }
    if (want || act != SP24_ACT_NONE)
        call("sp24_epilogue_backward", sp24_epilogue_backward, dY.data_ptr(), type, N, M, lddy, Z.t.defined() ? Z.t.data_ptr() : nullptr, Z.ld,
             static_cast<int>(act), act != SP24_ACT_NONE ? dZ.t.data_ptr() : nullptr, dZ.ld, want ? static_cast<float*>(dbias.data_ptr()) : nullptr,
             bytes ? work.data_ptr() : nullptr, stream_of(dY));
    return Py_BuildValue("(NN)", wrap(dZ.t), want ? wrap(dbias) : Py_NewRef(Py_None));
    END_HANDLE_TH_ERRORS
}

// Items of a list or tuple of the given length.
PyObject** items(PyObject* o, const char* name, Py_ssize_t n) {
    TORCH_CHECK_TYPE(PyList_Check(o) || PyTuple_Check(o), name, " must be a list or tuple");
    TORCH_CHECK_VALUE(PySequence_Fast_GET_SIZE(o) == n, name, " must hold ", n, " items, not ", PySequence_Fast_GET_SIZE(o));
    return PySequence_Fast_ITEMS(o);
}

void* flat(PyObject* o, const char* name, const Tensor& first, at::ScalarType type, at::IntArrayRef shape) {
    const Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.device() == first.device(), name, " must be on the first parameter's device");
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be of type ", type, ", not ", t.scalar_type());
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", not ", t.sizes());
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    return t.data_ptr();
}

const Tensor* device_scalar(PyObject* o, const char* name, const Tensor& first, at::ScalarType type) {
    if (is_none(o) || !THPVariable_Check(o)) return nullptr;
    const Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.device() == first.device() && t.scalar_type() == type && t.numel() == 1, name, " must be one ", type, " on the parameters' device");
    return &t;
}

// What a step writes of a tensor, each with the input that it may be.
std::array<std::pair<const void*, const void*>, 6> written_by(const sp24_adamw_tensor& t) {
    return {{{t.p_out, t.p}, {t.m_out, t.m}, {t.v_out, t.v}, {t.m_scales_out, t.m_scales}, {t.v_scales_out, t.v_scales}, {t.copy, nullptr}}};
}

// The written addresses of a step and their inputs, in a flat table: with a node for each a call of 100 tensors takes 30 us (8 bits 48), so
// 20 (23).
class Written {
    std::vector<std::pair<const void*, const void*>> slots;
    int shift;

public:
    explicit Written(size_t most) : shift(63) {
        while ((size_t{1} << (64 - shift)) < 2 * most) shift--;
        slots.resize(size_t{1} << (64 - shift));
    }
    // The slot of an address, or the free one that it would take.
    std::pair<const void*, const void*>& at(const void* x) {
        size_t i = static_cast<size_t>(reinterpret_cast<uintptr_t>(x) * 0x9E3779B97F4A7C15ull >> shift);
        while (slots[i].first != nullptr && slots[i].first != x) i = (i + 1) & (slots.size() - 1);
        return slots[i];
    }
};

// adamw(params, grads, states, step, lr, beta1, beta2, eps, weight_decay, grad_scale, seed, copies, params_out, states_out, first_index)
PyObject* adamw(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    SP24_ARGS(15);
    TORCH_CHECK_TYPE(PyList_Check(a[0]) || PyTuple_Check(a[0]), "params must be a list or tuple");
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(a[0]);
    const int64_t first_index = integer(a[14], "first_index");
    TORCH_CHECK_VALUE(first_index >= 0 && first_index <= (int64_t{1} << 32) - n, "first_index must be a place in the model below 2^32, not ", first_index);
    if (n == 0) Py_RETURN_NONE;
    PyObject** const P = PySequence_Fast_ITEMS(a[0]);
    PyObject** const G = items(a[1], "grads", n);
    PyObject** const S = items(a[2], "states", n);
    PyObject** const C = is_none(a[11]) ? nullptr : items(a[11], "copies", n);
    PyObject** const PO = is_none(a[12]) ? P : items(a[12], "the parameters of out", n);
    PyObject** const SO = is_none(a[13]) ? S : items(a[13], "the states of out", n);
    const Tensor& first = tensor(P[0], "a parameter");
    TORCH_CHECK_VALUE(first.is_cuda(), "sp24 operates on device tensors only");
    const c10::DeviceGuard guard(first.device());
    at::ScalarType grad = at::kFloat, copy = at::kBFloat16;
    bool any_grad = false, any_copy = false, bits8 = false;
    std::vector<sp24_adamw_tensor> list;
    list.reserve(n);
    Written written(6 * n);
    for (Py_ssize_t i = 0; i < n; i++) {
        if (is_none(G[i])) continue;  // no gradient: the tensor stays as it is
        const Tensor &p = tensor(P[i], "a parameter"), &g = tensor(G[i], "a gradient");
        if (!any_grad) {
            grad = g.scalar_type();
            float_type(g, "a gradient");
            TORCH_CHECK_TYPE(PyList_Check(S[i]) || PyTuple_Check(S[i]), "a state must be a list or tuple");
            bits8 = PySequence_Fast_GET_SIZE(S[i]) == 4;
        }
        any_grad = true;
        const auto shape = p.sizes();
        sp24_adamw_tensor t = {};
        t.n = p.numel();
        t.index = first_index + i;
        t.p = static_cast<const float*>(flat(P[i], "a parameter", first, at::kFloat, shape));
        t.p_out = static_cast<float*>(flat(PO[i], "a parameter of out", first, at::kFloat, shape));
        t.g = flat(G[i], "a gradient", first, grad, shape);
        const Py_ssize_t parts = bits8 ? 4 : 2;
        PyObject** const s = items(S[i], "a state", parts);
        PyObject** const so = items(SO[i], "a state of out", parts);
        if (bits8) {
            const std::array<int64_t, 1> nb{(t.n + 127) / 128};
            t.m = flat(s[0], "a first moment's codes", first, kCodes, shape);
            t.m_scales = static_cast<const uint8_t*>(flat(s[1], "a first moment's scales", first, kScales, nb));
            t.v = flat(s[2], "a second moment's codes", first, at::kByte, shape);
            t.v_scales = static_cast<const uint8_t*>(flat(s[3], "a second moment's scales", first, kScales, nb));
            t.m_out = flat(so[0], "a first moment's codes of out", first, kCodes, shape);
            t.m_scales_out = static_cast<uint8_t*>(flat(so[1], "a first moment's scales of out", first, kScales, nb));
            t.v_out = flat(so[2], "a second moment's codes of out", first, at::kByte, shape);
            t.v_scales_out = static_cast<uint8_t*>(flat(so[3], "a second moment's scales of out", first, kScales, nb));
        } else {
            t.m = flat(s[0], "a first moment", first, at::kFloat, shape);
            t.v = flat(s[1], "a second moment", first, at::kFloat, shape);
            t.m_out = flat(so[0], "a first moment of out", first, at::kFloat, shape);
            t.v_out = flat(so[1], "a second moment of out", first, at::kFloat, shape);
        }
        if (C && !is_none(C[i])) {
            if (!any_copy) {
                copy = tensor(C[i], "a copy").scalar_type();
                TORCH_CHECK_VALUE(copy == at::kBFloat16 || copy == at::kHalf, "copies must be bfloat16 or float16, not ", copy);
            }
            any_copy = true;
            t.copy = flat(C[i], "a copy", first, copy, shape);
        }
        if (t.n)
            for (const auto& [to, from] : written_by(t)) {
                if (to == nullptr) continue;
                auto& slot = written.at(to);
                TORCH_CHECK_VALUE(slot.first == nullptr, "a tensor is given twice");
                slot = {to, from};
            }
        list.push_back(t);
    }
    if (!any_grad) Py_RETURN_NONE;
    if (PO != P || SO != S)  // in place every input is what is written in its place
        for (const auto& t : list)
            for (const auto& [to, from] : written_by(t)) {
                if (from == nullptr || t.n == 0) continue;
                const auto& slot = written.at(from);
                TORCH_CHECK_VALUE(slot.first == nullptr || slot.second == from, "a tensor of out is the input of another");
            }
    const Tensor* const step_dev = device_scalar(a[3], "step", first, at::kLong);
    const Tensor* const lr_dev = device_scalar(a[4], "lr", first, at::kFloat);
    const Tensor* const scale = device_scalar(a[9], "grad_scale", first, at::kFloat);
    TORCH_CHECK_TYPE(is_none(a[9]) || scale, "grad_scale must be a tensor");
    const uint64_t seed = PyLong_AsUnsignedLongLongMask(a[10]);
    if (PyErr_Occurred()) throw python_error();
    Tensor work;
    if (step_dev || lr_dev) work = empty(16, at::kByte, first);
    call("sp24_adamw", sp24_adamw, list.data(), static_cast<int64_t>(list.size()),
         static_cast<int>(grad == at::kBFloat16 ? SP24_BF16 : grad == at::kHalf ? SP24_FP16 : SP24_FP32),
         static_cast<int>(bits8 ? SP24_FP8 : SP24_FP32), static_cast<int>(copy == at::kHalf ? SP24_FP16 : SP24_BF16),
         lr_dev ? 0.0 : number(a[4]), lr_dev ? static_cast<const float*>(lr_dev->data_ptr()) : nullptr, step_dev ? int64_t{0} : integer(a[3], "step"),
         step_dev ? static_cast<const int64_t*>(step_dev->data_ptr()) : nullptr, number(a[5]), number(a[6]), number(a[7]), number(a[8]),
         scale ? static_cast<const float*>(scale->data_ptr()) : nullptr, seed, work.defined() ? work.data_ptr() : nullptr, stream_of(first));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {SP24_METHOD(init), SP24_METHOD(gemm_bf16), SP24_METHOD(gemm_fp8), SP24_METHOD(epilogue_backward), SP24_METHOD(adamw),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_binding(void) { return PyModule_Create(&module); }
