// C ABI of the epilogue's gradient and the AdamW step, and the checks that the fused products share: argument validation
// (host only, before any HIP call), the device check, and the launches. Declarations and the contract live in
// include/sp24_layer.h.
#include "../../include/sp24.h"
#include "../../include/sp24_layer.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "adamw.h"
#include "sp24_launch.h"

namespace {

constexpr int64_t kMaxPitch = (int64_t)1 << 23, kMaxRows = ((int64_t)1 << 31) - 1, kMaxColumns = (int64_t)1 << 22;
constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;  // workgroups of 256 threads in one launch
constexpr int64_t kMaxElements = (int64_t)1 << 34;
constexpr double kLeastEps = 0x1p-126;  // the least normal fp32: the step multiplies by 1 / (sqrt(v) + eps), which has to be finite

bool aligned(const void* p, int to) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(to - 1)) == 0; }
bool is_float(int dt) { return dt == SP24_BF16 || dt == SP24_FP16 || dt == SP24_FP32; }
bool is_activation(int a) { return a == SP24_ACT_NONE || a == SP24_ACT_GELU || a == SP24_ACT_RELU || a == SP24_ACT_SILU; }
int hip_status(hipError_t e) { return e == hipSuccess ? SP24_OK : SP24_ERR_HIP; }
int check_size(int64_t N, int64_t M) { return N < 1 || N > kMaxRows || M < 1 || M > kMaxColumns ? SP24_ERR_SHAPE : SP24_OK; }

// An output of n elements that is its input or overlaps it nowhere.
bool apart(const void* in, const void* out, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
    return a == b || a + (uintptr_t)bytes <= b || b + (uintptr_t)bytes <= a;
}

int check_tensor(const sp24_adamw_tensor& t, bool bits8) {
    if (t.n < 0 || t.n > kMaxElements) return SP24_ERR_SHAPE;
    if (t.index < 0 || t.index > 0xFFFFFFFFll) return SP24_ERR_ARG;
    if (t.n == 0) return SP24_OK;
    if (!t.p || !t.p_out || !t.g || !t.m || !t.m_out || !t.v || !t.v_out) return SP24_ERR_NULL;
    if (bits8 && (!t.m_scales || !t.m_scales_out || !t.v_scales || !t.v_scales_out)) return SP24_ERR_NULL;
    if (!bits8 && (t.m_scales || t.m_scales_out || t.v_scales || t.v_scales_out)) return SP24_ERR_ARG;
    for (const void* p : {(const void*)t.p, (const void*)t.p_out, t.g, t.m, (const void*)t.m_out, t.v, (const void*)t.v_out, (const void*)t.copy})
        if (!aligned(p, 16)) return SP24_ERR_ALIGN;
    const int64_t state = bits8 ? t.n : 4 * t.n, blocks = (t.n + 127) / 128;
    if (!apart(t.p, t.p_out, 4 * t.n) || !apart(t.m, t.m_out, state) || !apart(t.v, t.v_out, state)) return SP24_ERR_ARG;
    if (bits8 && (!apart(t.m_scales, t.m_scales_out, blocks) || !apart(t.v_scales, t.v_scales_out, blocks))) return SP24_ERR_ARG;
    return SP24_OK;
}

bool finite_from_zero(double x) { return x >= 0.0 && x <= 3.402823466e+38; }

}  // namespace

namespace sp24 {

int check_epilogue(const float* bias, int activation, const void* R, int64_t ldr, const void* Z, int64_t ldz, const void* Y, int64_t ldy,
                   int64_t length) {
    if (!is_activation(activation)) return SP24_ERR_ARG;
    if ((R && ldr < length) || (Z && ldz < length)) return SP24_ERR_SHAPE;
    if (!aligned(bias, 4) || !aligned(R, 16) || !aligned(Z, 16)) return SP24_ERR_ALIGN;
    if ((R == Y && ldr != ldy) || Z == Y || (Z && Z == R)) return SP24_ERR_ARG;
    return SP24_OK;
}

}  // namespace sp24

extern "C" {

int sp24_epilogue_backward_bytes(int64_t N, int64_t M, int64_t* bytes) {
    if (!bytes) return SP24_ERR_NULL;
    const int st = check_size(N, M);
    if (st != SP24_OK) return st;
    const int parts = sp24::epilogue_back_parts(N, M);
    *bytes = parts > 1 ? (int64_t)parts * M * 4 : 0;
    return SP24_OK;
}

int sp24_epilogue_backward(const void* dY, int dtype, int64_t N, int64_t M, int64_t lddy, const void* Z, int64_t ldz,
                           int activation, void* dZ, int64_t lddz, float* dbias, void* workspace, void* stream) {
    if (!is_float(dtype)) return dY ? SP24_ERR_DTYPE : SP24_ERR_NULL;
    if (!is_activation(activation)) return SP24_ERR_ARG;
    const bool act = activation != SP24_ACT_NONE;
    if (!dY || (act && (!Z || !dZ)) || (!act && !dbias)) return SP24_ERR_NULL;
    if (!act && (Z || dZ)) return SP24_ERR_ARG;
    int st = check_size(N, M);
    if (st != SP24_OK) return st;
    if (lddy < M || lddy >= kMaxPitch || (act && (ldz < M || ldz >= kMaxPitch || lddz < M || lddz >= kMaxPitch))) return SP24_ERR_SHAPE;
    if (dbias && !workspace && sp24::epilogue_back_parts(N, M) > 1) return SP24_ERR_NULL;
    if (!aligned(dY, 16) || !aligned(Z, 16) || !aligned(dZ, 16) || !aligned(workspace, 16) || !aligned(dbias, 4)) return SP24_ERR_ALIGN;
    if (act && ((dZ == dY && lddz != lddy) || (dZ == Z && lddz != ldz))) return SP24_ERR_ARG;
    st = sp24::check_device();
    if (st != SP24_OK) return st;
    return hip_status(sp24::launch_epilogue_back(dY, dtype, N, M, lddy, Z, ldz, activation, dZ, lddz, dbias, workspace,
                                                 static_cast<hipStream_t>(stream)));
}

int sp24_adamw(const sp24_adamw_tensor* tensors, int64_t count, int grad_dtype, int state_dtype, int copy_dtype, double lr,
               const float* lr_dev, int64_t step, const int64_t* step_dev, double beta1, double beta2, double eps,
               double weight_decay, const float* grad_scale, uint64_t seed, void* workspace, void* stream) {
    if (count < 0 || count > 0x7FFFFFFF) return SP24_ERR_SHAPE;
    if (count && !tensors) return SP24_ERR_NULL;
    if (!is_float(grad_dtype) || (state_dtype != SP24_FP32 && state_dtype != SP24_FP8)) return SP24_ERR_DTYPE;
    if (copy_dtype != SP24_BF16 && copy_dtype != SP24_FP16) return SP24_ERR_DTYPE;
    const bool later = lr_dev || step_dev, bits8 = state_dtype == SP24_FP8;
    if (later && !workspace) return SP24_ERR_NULL;
    if (!later && workspace) return SP24_ERR_ARG;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= kLeastEps) || !finite_from_zero(eps)) return SP24_ERR_ARG;
    if ((!lr_dev && !finite_from_zero(lr)) || !finite_from_zero(weight_decay) || (!step_dev && step < 1)) return SP24_ERR_ARG;
    if (!aligned(lr_dev, 4) || !aligned(step_dev, 8) || !aligned(grad_scale, 4) || !aligned(workspace, 16)) return SP24_ERR_ALIGN;
    bool copies = false;
    for (int64_t i = 0; i < count; i++) {
        const int st = check_tensor(tensors[i], bits8);
        if (st != SP24_OK) return st;
        copies |= tensors[i].n && tensors[i].copy;
    }
    int st = sp24::check_device();
    if (st != SP24_OK) return st;

    const hipStream_t s = static_cast<hipStream_t>(stream);
    const sp24::AdamSchedule h{lr, beta1, beta2, weight_decay, lr_dev, step_dev, step, seed};
    sp24::AdamArgs a = {};
    a.b1 = (float)beta1, a.c1 = (float)(1.0 - beta1), a.b2 = (float)beta2, a.c2 = (float)(1.0 - beta2), a.eps = (float)eps;
    a.grad_scale = grad_scale;
    if (later) {
        a.later = static_cast<sp24::AdamScalars*>(workspace);
        st = hip_status(sp24::launch_adam_scalars(h, static_cast<sp24::AdamScalars*>(workspace), s));
        if (st != SP24_OK) return st;
    } else {
        a.now = sp24::adam_scalars(h);
    }
    int64_t blocks = 0;
    const auto flush = [&]() -> int {
        if (!a.count) return SP24_OK;
        const hipError_t e = sp24::launch_adamw(a, grad_dtype, bits8, copies ? copy_dtype : SP24_FP32, (unsigned)blocks, s);
        a.count = 0;
        blocks = 0;
        return hip_status(e);
    };
    for (int64_t i = 0; i < count; i++) {
        const sp24_adamw_tensor& t = tensors[i];
        if (!t.n) continue;
        const int64_t mine = (t.n + sp24::ADAM_CHUNK - 1) / sp24::ADAM_CHUNK;
        if (a.count == sp24::ADAM_TENSORS || blocks + mine > kMaxGrid) {
            st = flush();
            if (st != SP24_OK) return st;
        }
        sp24::AdamTensor& d = a.t[a.count];
        d.p = t.p, d.p_out = t.p_out, d.g = static_cast<const char*>(t.g);
        d.m = static_cast<const char*>(t.m), d.m_out = static_cast<char*>(t.m_out);
        d.v = static_cast<const char*>(t.v), d.v_out = static_cast<char*>(t.v_out);
        d.ms = t.m_scales, d.ms_out = t.m_scales_out, d.vs = t.v_scales, d.vs_out = t.v_scales_out;
        d.copy = static_cast<char*>(t.copy), d.n = t.n, d.index = (uint32_t)t.index;
        a.first[a.count++] = (uint32_t)blocks;
        blocks += mine;
    }
    return flush();
}

}  // extern "C"
