/*
 * sp24, 8-bit floating point -- activations and 2:4 weights held in 8 bits with a scale for each block of 128,
 * the operators that make, use and differentiate them around a Linear layer, for AMD MI355X (gfx950).
 *
 * Format:
 *  codes   OCP e4m3 (bias 7, largest finite 448, 0x7F / 0xFF NaN).
 *  scales  one byte s for each block, the power of two 2^(s - 127) (OCP e8m0; 0xFF is NaN). A code's value is
 *          code * 2^(s - 127): 4 significant bits, so also exactly a bf16 number wherever that is in bf16's range.
 *  activations: N x K tokens x channels, codes row-major with pitch ldc bytes; a block is 128 consecutive
 *          channels of a token (the last one of a row is shorter where K is no multiple of 128); the scale of
 *          channels 128 b .. of token n is scales[n * lds + b], lds >= ceil(K / 128).
 *  weights: M x K, 2:4 along K, values (e4m3) and meta in the tiled layout of sp24.h for 1-byte values; a block
 *          is 128 x 128, its scale w_scales[(m / 128) * ceil(K / 128) + k / 128].
 *  A block's scale is the least power of two (at least 2^-127) that keeps its largest magnitude within 448 units;
 *  its codes are the values times 2^(127 - s), rounded once to nearest even. A block of an activation that holds an
 *  infinity or a NaN gets the scale NaN, so that every value in it reads as NaN; its codes are then unspecified.
 *
 * Conventions are those of sp24.h (caller-owned device memory, asynchronous on `stream`, validated on the host
 * before any launch, K a positive multiple of 16, M, N >= 1). In addition: base pointers of matrices are 16-byte
 * aligned; a pitch in bytes is a multiple of 16, except that of an output Y (any pitch) and of scales; pitches are
 * below 2^23 elements, those of scales below 2^22; K is at most 2^20, N below 2^31, M at most 2^22 (what would need
 * 2^32 threads or more in one launch is SP24_ERR_SHAPE). Results are deterministic: no sum depends on the order in
 * which workgroups run.
 */
#ifndef SP24_FP8_H
#define SP24_FP8_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* X (N x K of dtype BF16, FP16 or FP32, pitch ldx) as codes and scales: the input of sp24_gemm_fp8 where no norm
 * precedes it, and the 8-bit copy of an activation that sp24_grad_weight_fp8 reads in the backward pass. */
int sp24_quant_fp8(const void* X, int dtype, int64_t N, int64_t K, int64_t ldx, uint8_t* codes, int64_t ldc,
                   uint8_t* scales, int64_t lds, void* stream);

/* Root-mean-square norm with the residual's addition and an 8-bit output:
 *   h = X + R, rounded to dtype (R == NULL: h = X),  r = 1 / sqrt(mean_k h^2 + eps),  y = h * r * gamma,
 *   codes, scales = y in the format above.
 *   X, R, H: N x K of dtype (BF16, FP16 or FP32); gamma: K of dtype. H receives h: required with R and NULL
 *   without; it may be X or R themselves (same base and pitch). rstd: fp32[N] receives r, or NULL. eps >= 0, and
 *   a row of zeros with eps == 0 gives NaN. K <= 32768. The mean is held in fp32. */
int sp24_rmsnorm_fp8(const void* X, int dtype, int64_t N, int64_t K, int64_t ldx, const void* R, int64_t ldr,
                     const void* gamma, float eps, void* H, int64_t ldh, uint8_t* codes, int64_t ldc, uint8_t* scales,
                     int64_t lds, float* rstd, void* stream);

/* Gradients of the norm, from dY (the gradient of y; rounding to codes is passed straight through) and dH (the
 * gradient of h from the residual stream, or NULL):
 *   xhat = h * r,  c = mean_k(gamma * dY * xhat),  dX = r * (gamma * dY - xhat * c) + dH,
 *   dgamma[k] = sum_n dY * xhat  (fp32[K]).
 * dX is the gradient of X and of R alike. dY, H, dH, dX: N x K of dtype; dX may be dY or dH themselves. rstd is
 * what sp24_rmsnorm_fp8 returned. K <= 32768. workspace: sp24_rmsnorm_backward_bytes(N, K) bytes, 16-byte aligned
 * (partial sums of dgamma, added in a fixed order). */
int sp24_rmsnorm_backward_bytes(int64_t N, int64_t K, int64_t* bytes);
int sp24_rmsnorm_backward(const void* dY, int dtype, int64_t N, int64_t K, int64_t lddy, const void* H, int64_t ldh,
                          const float* rstd, const void* gamma, const void* dH, int64_t lddh, void* dX, int64_t lddx,
                          float* dgamma, void* workspace, void* stream);

/* 2:4 prune and compress W (M x K of dtype BF16, FP16 or FP32, pitch ldw; selection as sp24_prune_compress) to e4m3
 * values with a scale for each 128 x 128 block of kept values. values and meta: the sizes that
 * sp24_compressed_bytes gives for SP24_FP8; w_scales: ceil(M / 128) * ceil(K / 128) bytes. Inputs must be finite. */
int sp24_prune_compress_fp8(const void* W, int dtype, int64_t M, int64_t K, int64_t ldw, int score, const float* norms,
                            uint8_t* values, uint8_t* meta, uint8_t* w_scales, void* stream);

/* The dense weight back as out_dtype BF16 or FP32 (exact wherever it is in that type's range), +0 at pruned places:
 * the operand of the input's gradient, dX = dY * W, which is no 2:4 product (the sum runs over M). */
int sp24_decompress_fp8(const uint8_t* values, const uint8_t* meta, const uint8_t* w_scales, int64_t M, int64_t K,
                        void* W_out, int out_dtype, int64_t ldw, void* stream);

/* 2:4 sparse x dense product in 8-bit floating point with a scale for each block of 128:
 *   Y[n, m] = sum_b 2^(x_scales[n, b] + w_scales[m / 128, b] - 254) * sum_{kept k in block b} w[m, k] * x[n, k],
 *   sums over blocks in fp32, Y: N x M (pitch ldy >= M) of out_dtype BF16 or FP16 (rounded once; FP16 overflows to
 *   infinity). X codes: N x K, pitch ldx. Inside a block the 8-bit matrix instructions align the 64 products to about
 *   2^-13 of the largest one (measured): far below the codes' own 2^-4, and by norm below the rounding to 16 bits, but a
 *   single result whose products cancel can be off by more than that rounding. An FP32 result would promise more, so
 *   none is offered.
 * A NaN scale of x makes its token's row NaN, one of the weight its 128 output channels. The product of two scales
 * must be below 2^128; one below 2^-149 may count as zero. Results depend on the sizes, which choose the kernel, only
 * through the order of the fp32 sums, however far apart a token's scales are. */
int sp24_gemm_fp8(const uint8_t* values, const uint8_t* meta, const uint8_t* w_scales, int64_t M, int64_t K,
                  const uint8_t* X, int64_t N, int64_t ldx, const uint8_t* x_scales, int64_t lds, void* Y, int out_dtype,
                  int64_t ldy, void* stream);

/* Gradient of the weight of Y = X W^T from the 8-bit copy of X:
 *   dW[m, k] = sum_n dY[n, m] * x[n, k] * 2^(x_scales[n, k / 128] - 127),  products exact, sums in fp32.
 *   dY: bf16 N x M (pitch lddy); X, x_scales: N x K codes and scales; dW: M x K (pitch ldw) of out_dtype FP32 or
 *   BF16 (rounded once). meta: NULL, or the metadata of an M x K weight with 1-byte values: then dW is +0 at the
 *   pruned places (training the kept weights only). workspace: sp24_grad_weight_fp8_bytes(M, K, N) bytes (may be 0:
 *   then NULL), 16-byte aligned: partial sums over tokens where the weight alone gives too few tiles. */
int sp24_grad_weight_fp8_bytes(int64_t M, int64_t K, int64_t N, int64_t* bytes);
int sp24_grad_weight_fp8(const void* dY, int64_t N, int64_t M, int64_t lddy, const uint8_t* X, int64_t K, int64_t ldx,
                         const uint8_t* x_scales, int64_t lds, const uint8_t* meta, void* dW, int out_dtype, int64_t ldw,
                         void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SP24_FP8_H */
