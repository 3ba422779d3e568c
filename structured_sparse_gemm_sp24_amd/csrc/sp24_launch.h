// Host-side launchers of the sp24 kernels (internal to the library; the C ABI in sp24_api.cpp
// validates arguments before calling these).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sp24 {

// Output kinds of the int8 GEMM.
enum OutKind { OUT_I32 = 0, OUT_F32 = 1, OUT_BF16 = 2, OUT_I8 = 3 };

// Operands of one sparse GEMM call, validated by the C ABI. Element strides are in elements of the
// operand's type.
//   feature-major (tm == false): X is K x N (X[k, n] at k * ldx + n), Y is M x N (Y[m, n] at m * ldy + n)
//   token-major   (tm == true):  X is N x K (X[k, n] at n * ldx + k), Y is N x M (Y[m, n] at n * ldy + m)
//   batch b (0 <= b < batch) adds b * sx to X and b * sy to Y; the weight is shared.
struct GemmArgs {
    const void* values;
    const uint8_t* meta;
    int64_t M, K, N;
    const void* X;
    int64_t ldx, sx;
    void* Y;
    int64_t ldy, sy;
    int64_t batch;
    bool tm;
    const float* scale;  // int8 only: per-row dequant scale, or NULL for raw int32 output
    bool out_fp32;       // bf16 only: fp32 output (else bf16)
    // int8 epilogue (with scale): y = fl32(fl32(acc) * scale[m]), + bias[m] when bias is set, GELU when
    // gelu is set, then stored as out_kind (OUT_F32, OUT_BF16 round to nearest even, OUT_I8
    // clamp(rne(fl32(y * inv_scale)), -127, 127)); without scale out_kind is OUT_I32 (raw accumulators)
    const float* bias;
    int gelu;
    int out_kind;
    float inv_scale;
};

hipError_t launch_col_norms(const uint16_t* X, int64_t K, int64_t N, int64_t ldx, float* norms, hipStream_t s);

hipError_t launch_prune_compress(const void* W, int dtype, int64_t M, int64_t K, int64_t ldw, int score,
                                 const float* norms, void* values, int val_dtype, uint8_t* meta, hipStream_t s);

hipError_t launch_prune_mask(const void* W, int dtype, int64_t M, int64_t K, int64_t ldw, int keep, int score,
                             const float* norms, uint8_t* mask, void* W_out, int64_t ldo, hipStream_t s);

// Shader-clock probe: `blocks` workgroups of 4 waves, cycles and real-time ticks per wave into out.
hipError_t launch_sclk_probe(int64_t blocks, int iters, uint64_t* out, hipStream_t s);
hipError_t launch_channel_permutation(const void* W, int dtype, int64_t M, int64_t K, int64_t ldw, int score,
                                      const float* norms, int sweeps, int32_t* perm, hipStream_t s);

hipError_t launch_decompress(const void* values, const uint8_t* meta, int dtype, int64_t M, int64_t K,
                             void* W_out, int64_t ldw, hipStream_t s);

// bf16 GEMM: the kernel is chosen from the shape, layout and alignment (few tokens, LDS-tiled, direct).
hipError_t launch_gemm_bf16(const GemmArgs& g, hipStream_t s);
bool gemm_bf16_skinny_ok(const GemmArgs& g);
hipError_t launch_gemm_bf16_skinny(const GemmArgs& g, hipStream_t s);
// Compute units of the current device (cached per device; 256 if the query fails).
int device_cus();
// Workgroup tile width (256, or 128 for token-major X) of a tiled int8 GEMM launch.
int tiled_tile_width(const GemmArgs& g);
// Few-token GEMM in the Linear layout (token-major, N <= 16) with the weight streamed through LDS.
bool gemm_bf16_fewtok_ok(const GemmArgs& g);
hipError_t launch_gemm_bf16_fewtok(const GemmArgs& g, hipStream_t s);
bool gemm_bf16_tiled_ok(const GemmArgs& g);
hipError_t launch_gemm_bf16_tiled(const GemmArgs& g, hipStream_t s);

// Dense reference with the token-major tiled kernel's tiling (measurement only): the weight converted to the
// MFMA operand order, and the GEMM (token-major X, batch 1; values = the converted weight).
hipError_t launch_dense_tile(const void* W, int64_t M, int64_t K, int64_t ldw, void* Wt, hipStream_t s);
hipError_t launch_gemm_dense_ref(const GemmArgs& g, hipStream_t s);

// Streaming read (measurement only): workgroups used for `bytes`, and the launch.
int stream_read_blocks(int64_t bytes);
hipError_t launch_stream_read(const void* src, int64_t bytes, void* sink, hipStream_t s);

// int8 GEMM: LDS-tiled when it applies, else direct.
hipError_t launch_gemm_i8(const GemmArgs& g, hipStream_t s);
bool gemm_i8_fewtok_ok(const GemmArgs& g);
hipError_t launch_gemm_i8_fewtok(const GemmArgs& g, hipStream_t s);
bool gemm_i8_tiled_ok(const GemmArgs& g);
hipError_t launch_gemm_i8_tiled(const GemmArgs& g, hipStream_t s);

// SP24_OK if the current device is gfx950, else SP24_ERR_DEVICE (sp24_api.cpp; cached per device).
int check_device();

// 8-bit floating point (include/sp24_fp8.h). dtype: 0 BF16, 1 FP16, 2 FP32 (the sp24_dtype numbers).
hipError_t launch_quant_fp8(const void* X, int dtype, int64_t N, int64_t K, int64_t ldx, uint8_t* codes, int64_t ldc,
                            uint8_t* scales, int64_t lds, hipStream_t s);
hipError_t launch_rmsnorm(const void* X, int dtype, int64_t N, int64_t K, int64_t ldx, const void* R, int64_t ldr,
                          const void* gamma, float eps, void* H, int64_t ldh, uint8_t* codes, int64_t ldc,
                          uint8_t* scales, int64_t lds, float* rstd, hipStream_t s);
// Rows of K partial sums that the norm's gradient writes to its workspace.
int rmsnorm_back_parts(int64_t N, int64_t K);
hipError_t launch_rmsnorm_back(const void* dY, int dtype, int64_t N, int64_t K, int64_t lddy, const void* H, int64_t ldh,
                               const float* rstd, const void* gamma, const void* dH, int64_t lddh, void* dX,
                               int64_t lddx, float* dgamma, void* workspace, hipStream_t s);
hipError_t launch_prune_compress_fp8(const void* W, int dtype, int64_t M, int64_t K, int64_t ldw, int score,
                                     const float* norms, uint8_t* values, uint8_t* meta, uint8_t* w_scales,
                                     hipStream_t s);
hipError_t launch_decompress_fp8(const uint8_t* values, const uint8_t* meta, const uint8_t* w_scales, int64_t M,
                                 int64_t K, void* W, bool f32, int64_t ldw, hipStream_t s);

// Token-major product with block scales: X N x K codes, Y N x M.
struct Fp8GemmArgs {
    const uint8_t *values, *meta, *ws, *X, *xs;
    void* Y;
    int64_t M, K, N, ldx, lds, ldy;
    bool out_fp16;  // else bf16
};
hipError_t launch_gemm_fp8(const Fp8GemmArgs& g, hipStream_t s);
hipError_t launch_gemm_fp8_tiled(const Fp8GemmArgs& g, hipStream_t s);

// Weight gradient: dY N x M bf16, X N x K codes, dW M x K; meta NULL or the 2:4 pattern of dW.
struct Fp8GradArgs {
    const void* dY;
    const uint8_t *X, *xs, *meta;
    void *dW, *workspace;
    int64_t N, M, K, lddy, ldx, lds, ldw;
    bool out_fp32;
};
// Parts that the tokens are split into; with more than one the workspace holds an M x K fp32 matrix for each.
int grad_weight_parts(int64_t M, int64_t K, int64_t N);
hipError_t launch_grad_weight(const Fp8GradArgs& g, hipStream_t s);
hipError_t launch_grad_weight_tiled(const Fp8GradArgs& g, hipStream_t s);

}  // namespace sp24
