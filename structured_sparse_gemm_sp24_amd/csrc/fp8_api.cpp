// C ABI of the 8-bit floating-point operators: argument validation (host only, before any HIP call), the device
// check, and the launches. Declarations and the contract live in include/sp24_fp8.h.
#include "../../include/sp24.h"
#include "../../include/sp24_fp8.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sp24_launch.h"

namespace {

constexpr int64_t kMaxPitch = (int64_t)1 << 23;   // elements: 64 rows of any type stay within 32-bit byte offsets
constexpr int64_t kMaxScalePitch = (int64_t)1 << 22;  // 256 rows likewise
constexpr int64_t kMaxK = (int64_t)1 << 20, kMaxNormK = 32768;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxWeightRows = (int64_t)1 << 22;
constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;  // workgroups of 256 threads in one launch

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool is_float(int dt) { return dt == SP24_BF16 || dt == SP24_FP16 || dt == SP24_FP32; }
int type_size(int dt) { return dt == SP24_FP32 ? 4 : 2; }
int64_t blocks_of(int64_t n) { return (n + 127) / 128; }
int64_t tiles_256(int64_t a, int64_t b) { return ((a + 255) / 256) * ((b + 255) / 256); }

int check_nk(int64_t N, int64_t K, int64_t most_k) {
    return N < 1 || N > kMaxRows || K < 16 || K % 16 != 0 || K > most_k ? SP24_ERR_SHAPE : SP24_OK;
}
// A row-major matrix with rows of `cols` elements of `es` bytes.
int check_matrix(const void* p, int64_t cols, int64_t ld, int es) {
    if (ld < cols || ld >= kMaxPitch) return SP24_ERR_SHAPE;
    return aligned16(p) && (ld * es) % 16 == 0 ? SP24_OK : SP24_ERR_ALIGN;
}
int check_scales(int64_t K, int64_t lds) { return lds < blocks_of(K) || lds >= kMaxScalePitch ? SP24_ERR_SHAPE : SP24_OK; }

int hip_status(hipError_t e) { return e == hipSuccess ? SP24_OK : SP24_ERR_HIP; }

#define SP24_TRY(call)                  \
    do {                                \
        const int st_ = (call);         \
        if (st_ != SP24_OK) return st_; \
    } while (0)

}  // namespace

extern "C" {

int sp24_quant_fp8(const void* X, int dtype, int64_t N, int64_t K, int64_t ldx, uint8_t* codes, int64_t ldc,
                   uint8_t* scales, int64_t lds, void* stream) {
    if (!X || !codes || !scales) return SP24_ERR_NULL;
    if (!is_float(dtype)) return SP24_ERR_DTYPE;
    SP24_TRY(check_nk(N, K, kMaxK));
    SP24_TRY(check_matrix(X, K, ldx, type_size(dtype)));
    SP24_TRY(check_matrix(codes, K, ldc, 1));
    SP24_TRY(check_scales(K, lds));
    SP24_TRY(sp24::check_device());
    return hip_status(sp24::launch_quant_fp8(X, dtype, N, K, ldx, codes, ldc, scales, lds, static_cast<hipStream_t>(stream)));
}

int sp24_rmsnorm_fp8(const void* X, int dtype, int64_t N, int64_t K, int64_t ldx, const void* R, int64_t ldr,
                     const void* gamma, float eps, void* H, int64_t ldh, uint8_t* codes, int64_t ldc, uint8_t* scales,
                     int64_t lds, float* rstd, void* stream) {
    if (!X || !gamma || !codes || !scales || (R && !H)) return SP24_ERR_NULL;
    if (!is_float(dtype)) return SP24_ERR_DTYPE;
    if (!R && H) return SP24_ERR_ARG;
    if (!(eps >= 0.f) || eps > 3.402823466e+38f) return SP24_ERR_ARG;
    SP24_TRY(check_nk(N, K, kMaxNormK));
    const int es = type_size(dtype);
    SP24_TRY(check_matrix(X, K, ldx, es));
    if (R) {
        SP24_TRY(check_matrix(R, K, ldr, es));
        SP24_TRY(check_matrix(H, K, ldh, es));
    }
    SP24_TRY(check_matrix(codes, K, ldc, 1));
    SP24_TRY(check_scales(K, lds));
    if (!aligned16(gamma) || (reinterpret_cast<uintptr_t>(rstd) & 3) != 0) return SP24_ERR_ALIGN;
    SP24_TRY(sp24::check_device());
    return hip_status(sp24::launch_rmsnorm(X, dtype, N, K, ldx, R, ldr, gamma, eps, H, ldh, codes, ldc, scales, lds, rstd,
                                           static_cast<hipStream_t>(stream)));
}

int sp24_rmsnorm_backward_bytes(int64_t N, int64_t K, int64_t* bytes) {
    if (!bytes) return SP24_ERR_NULL;
    SP24_TRY(check_nk(N, K, kMaxNormK));
    *bytes = (int64_t)sp24::rmsnorm_back_parts(N, K) * K * 4;
    return SP24_OK;
}

int sp24_rmsnorm_backward(const void* dY, int dtype, int64_t N, int64_t K, int64_t lddy, const void* H, int64_t ldh,
                          const float* rstd, const void* gamma, const void* dH, int64_t lddh, void* dX, int64_t lddx,
                          float* dgamma, void* workspace, void* stream) {
    if (!dY || !H || !rstd || !gamma || !dX || !dgamma || !workspace) return SP24_ERR_NULL;
    if (!is_float(dtype)) return SP24_ERR_DTYPE;
    SP24_TRY(check_nk(N, K, kMaxNormK));
    const int es = type_size(dtype);
    SP24_TRY(check_matrix(dY, K, lddy, es));
    SP24_TRY(check_matrix(H, K, ldh, es));
    if (dH) SP24_TRY(check_matrix(dH, K, lddh, es));
    SP24_TRY(check_matrix(dX, K, lddx, es));
    if (!aligned16(gamma) || !aligned16(workspace)) return SP24_ERR_ALIGN;
    if (((reinterpret_cast<uintptr_t>(rstd) | reinterpret_cast<uintptr_t>(dgamma)) & 3) != 0) return SP24_ERR_ALIGN;
    SP24_TRY(sp24::check_device());
    return hip_status(sp24::launch_rmsnorm_back(dY, dtype, N, K, lddy, H, ldh, rstd, gamma, dH, lddh, dX, lddx, dgamma,
                                                workspace, static_cast<hipStream_t>(stream)));
}

int sp24_prune_compress_fp8(const void* W, int dtype, int64_t M, int64_t K, int64_t ldw, int score, const float* norms,
                            uint8_t* values, uint8_t* meta, uint8_t* w_scales, void* stream) {
    if (!W || !values || !meta || !w_scales) return SP24_ERR_NULL;
    if (!is_float(dtype)) return SP24_ERR_DTYPE;
    if (score != SP24_SCORE_MAGNITUDE && score != SP24_SCORE_WANDA) return SP24_ERR_ARG;
    if (score == SP24_SCORE_WANDA && !norms) return SP24_ERR_NULL;
    if (score == SP24_SCORE_MAGNITUDE && norms) return SP24_ERR_ARG;
    SP24_TRY(check_nk(M, K, kMaxK));
    if (M > kMaxWeightRows || blocks_of(M) * blocks_of(K) > kMaxGrid / 2) return SP24_ERR_SHAPE;  // 512 threads
    SP24_TRY(check_matrix(W, K, ldw, type_size(dtype)));
    if (!aligned16(values) || !aligned16(meta) || (norms && !aligned16(norms))) return SP24_ERR_ALIGN;
    SP24_TRY(sp24::check_device());
    return hip_status(sp24::launch_prune_compress_fp8(W, dtype, M, K, ldw, score, norms, values, meta, w_scales,
                                                      static_cast<hipStream_t>(stream)));
}

int sp24_decompress_fp8(const uint8_t* values, const uint8_t* meta, const uint8_t* w_scales, int64_t M, int64_t K,
                        void* W_out, int out_dtype, int64_t ldw, void* stream) {
    if (!values || !meta || !w_scales || !W_out) return SP24_ERR_NULL;
    if (out_dtype != SP24_BF16 && out_dtype != SP24_FP32) return SP24_ERR_DTYPE;
    SP24_TRY(check_nk(M, K, kMaxK));
    if (M > kMaxWeightRows || (M + 15) / 16 * ((blocks_of(K) + 3) / 4) > kMaxGrid) return SP24_ERR_SHAPE;
    SP24_TRY(check_matrix(W_out, K, ldw, type_size(out_dtype)));
    if (!aligned16(values) || !aligned16(meta)) return SP24_ERR_ALIGN;
    SP24_TRY(sp24::check_device());
    return hip_status(sp24::launch_decompress_fp8(values, meta, w_scales, M, K, W_out, out_dtype == SP24_FP32, ldw,
                                                  static_cast<hipStream_t>(stream)));
}

int sp24_gemm_fp8(const uint8_t* values, const uint8_t* meta, const uint8_t* w_scales, int64_t M, int64_t K,
                  const uint8_t* X, int64_t N, int64_t ldx, const uint8_t* x_scales, int64_t lds, void* Y, int out_dtype,
                  int64_t ldy, void* stream) {
    if (!values || !meta || !w_scales || !X || !x_scales || !Y) return SP24_ERR_NULL;
    if (out_dtype != SP24_BF16 && out_dtype != SP24_FP16) return SP24_ERR_DTYPE;
    SP24_TRY(check_nk(N, K, kMaxK));
    if (M < 1 || M > kMaxWeightRows) return SP24_ERR_SHAPE;
    // tiles of 256 x 128 with 256 threads or of 256 x 256 with 512: one workgroup each where K is a single block
    if (((M + 255) / 256) * blocks_of(N) > kMaxGrid || tiles_256(M, N) > kMaxGrid / 2) return SP24_ERR_SHAPE;
    SP24_TRY(check_matrix(X, K, ldx, 1));
    SP24_TRY(check_scales(K, lds));
    if (ldy < M || ldy >= kMaxPitch) return SP24_ERR_SHAPE;
    if (!aligned16(values) || !aligned16(meta) || !aligned16(Y)) return SP24_ERR_ALIGN;
    SP24_TRY(sp24::check_device());
    sp24::Fp8GemmArgs g;
    g.values = values; g.meta = meta; g.ws = w_scales; g.X = X; g.xs = x_scales; g.Y = Y;
    g.M = M; g.K = K; g.N = N; g.ldx = ldx; g.lds = lds; g.ldy = ldy;
    g.out_fp16 = out_dtype == SP24_FP16;
    return hip_status(sp24::launch_gemm_fp8(g, static_cast<hipStream_t>(stream)));
}

int sp24_grad_weight_fp8_bytes(int64_t M, int64_t K, int64_t N, int64_t* bytes) {
    if (!bytes) return SP24_ERR_NULL;
    SP24_TRY(check_nk(N, K, kMaxK));
    if (M < 1 || M > kMaxWeightRows || tiles_256(M, K) > kMaxGrid / 2) return SP24_ERR_SHAPE;
    const int parts = sp24::grad_weight_parts(M, K, N);
    *bytes = parts > 1 ? (int64_t)parts * M * K * 4 : 0;
    return SP24_OK;
}

int sp24_grad_weight_fp8(const void* dY, int64_t N, int64_t M, int64_t lddy, const uint8_t* X, int64_t K, int64_t ldx,
                         const uint8_t* x_scales, int64_t lds, const uint8_t* meta, void* dW, int out_dtype, int64_t ldw,
                         void* workspace, void* stream) {
    if (!dY || !X || !x_scales || !dW) return SP24_ERR_NULL;
    if (out_dtype != SP24_BF16 && out_dtype != SP24_FP32) return SP24_ERR_DTYPE;
    SP24_TRY(check_nk(N, K, kMaxK));
    // one workgroup of 512 threads a tile (small weights, far below the limit, take smaller tiles)
    if (M < 1 || M > kMaxWeightRows || tiles_256(M, K) > kMaxGrid / 2) return SP24_ERR_SHAPE;
    if (!workspace && sp24::grad_weight_parts(M, K, N) > 1) return SP24_ERR_NULL;
    SP24_TRY(check_matrix(dY, M, lddy, 2));
    SP24_TRY(check_matrix(X, K, ldx, 1));
    SP24_TRY(check_scales(K, lds));
    SP24_TRY(check_matrix(dW, K, ldw, type_size(out_dtype)));
    if ((meta && !aligned16(meta)) || (workspace && !aligned16(workspace))) return SP24_ERR_ALIGN;
    SP24_TRY(sp24::check_device());
    sp24::Fp8GradArgs g;
    g.dY = dY; g.X = X; g.xs = x_scales; g.meta = meta; g.dW = dW; g.workspace = workspace;
    g.N = N; g.M = M; g.K = K; g.lddy = lddy; g.ldx = ldx; g.lds = lds; g.ldw = ldw;
    g.out_fp32 = out_dtype == SP24_FP32;
    return hip_status(sp24::launch_grad_weight(g, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
