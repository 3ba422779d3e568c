/*
 * sp24, layer operators -- what surrounds the 2:4 product in a Linear layer and trains it: products with bias,
 * activation and residual in their epilogue, that epilogue's gradient, and an AdamW step over many tensors, for AMD
 * MI355X (gfx950).
 *
 * Conventions are those of sp24.h (caller-owned device memory, asynchronous on `stream`, validated on the host before
 * any launch; results are deterministic). All entry points may be captured into a graph.
 *
 * Epilogue of the products, each step in fp32, acc being what the plain product sums:
 *   z = acc + bias[m]                       (bias: fp32[M], or NULL)
 *   y = act(z)                              (sp24_activation)
 *   y = y + R[n, m]                         (R: of Y's type and shape, or NULL)
 *   Y = round(y),  Z = round(z)             (Z: of Y's type and shape, for the backward pass, or NULL)
 *   GELU(z) = z Phi(z) as in sp24_gemm_i8_fused, |error| <= 8 * 2^-24 |z|; SiLU(z) = z / (1 + e^-z), within
 *   (6 + 3 |z|) * 2^-24 of itself (z >= -87); ReLU(z) = max(z, 0). Infinities have their limits, NaN stays NaN.
 * R and Z have a base aligned to 16 bytes and any pitch of at least a row. R may be Y (same base, pitch and batch
 * stride: each element is read before it is written) and shares no element with it otherwise; Z shares none with either.
 */
#ifndef SP24_LAYER_H
#define SP24_LAYER_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* sp24_gemm_bf16_ex with the epilogue above. R, Z and Y in the layout of Y (feature-major M x N, token-major N x M), batch
 * entries their strides apart: r_batch_stride >= 0 (0: one residual for all), z_batch_stride at least one entry's
 * extent, both multiples of 16 bytes and ignored with batch == 1. */
int sp24_gemm_bf16_fused(const void* values, const uint8_t* meta, int64_t M, int64_t K, const void* X, int64_t N, int64_t ldx,
                         int64_t x_batch_stride, const float* bias, int activation, const void* R, int64_t ldr,
                         int64_t r_batch_stride, void* Z, int64_t ldz, int64_t z_batch_stride, void* Y, int out_dtype,
                         int64_t ldy, int64_t y_batch_stride, int64_t batch, int layout, void* stream);

/* sp24_gemm_fp8 with the epilogue above (token-major: R, Z and Y are N x M). A NaN scale makes its outputs NaN with every
 * activation. */
int sp24_gemm_fp8_fused(const uint8_t* values, const uint8_t* meta, const uint8_t* w_scales, int64_t M, int64_t K,
                        const uint8_t* X, int64_t N, int64_t ldx, const uint8_t* x_scales, int64_t lds, const float* bias,
                        int activation, const void* R, int64_t ldr, void* Z, int64_t ldz, void* Y, int out_dtype, int64_t ldy,
                        void* stream);

/* Gradients of the epilogue (token-major) from dY, that of Y, and the Z that the product kept:
 *   dZ[n, m] = dY[n, m] act'(Z[n, m]),  dbias[m] = sum_n dY[n, m] act'(Z[n, m])  (fp32[M], from unrounded products).
 * dZ is what sp24_grad_weight_fp8 and the input's gradient take; the residual's gradient is dY itself. ReLU' is 1 where
 * Z > 0 and chooses: dZ is +0 elsewhere whatever dY holds.
 * Of a feature-major product's Z (M x N, an entry a call) this gives dZ alone: rows are then channels, dbias would be a sum
 * over channels and is left NULL, and the bias's gradient, one along rows, is not offered.
 *   dY, Z, dZ: N x M of dtype (BF16, FP16 or FP32), base 16-byte aligned, any pitch of at least M and below 2^23. dZ may be
 *   dY or Z (same base and pitch). dbias: NULL where there is no bias. With SP24_ACT_NONE dZ would be dY: Z and dZ must
 *   be NULL and dbias not. N below 2^31, M at most 2^22. workspace: sp24_epilogue_backward_bytes(N, M) bytes (may be
 *   0: then NULL), 16-byte aligned: partial sums of dbias, added in a fixed order; not read without dbias. */
int sp24_epilogue_backward_bytes(int64_t N, int64_t M, int64_t* bytes);
int sp24_epilogue_backward(const void* dY, int dtype, int64_t N, int64_t M, int64_t lddy, const void* Z, int64_t ldz,
                           int activation, void* dZ, int64_t lddz, float* dbias, void* workspace, void* stream);

/* One tensor of an AdamW step. Every pointer to elements is 16-byte aligned; each *_out is the tensor beside it (in place) or
 * memory that overlaps nothing else. With n == 0 the tensor is passed over.
 *  32-bit states: m, v fp32[n]; the scales are NULL.
 *  8-bit states, a block being 128 consecutive elements (the last one shorter):
 *    first moment:  m uint8[n] e4m3 codes, m_scales uint8[ceil(n / 128)]: m = code * 2^(s - 127), the format of sp24_fp8.h;
 *    second moment: v uint8[n] whole numbers c, v_scales uint8[ceil(n / 128)]: v = (c * 2^(s - 127))^2, s at least 64, the
 *      least that keeps the block's largest root within 255 units.
 *    Zeroed bytes are a state of zeros. An infinite or NaN moment makes its block's scale 255, and the block NaN for good. */
typedef struct {
    const float* p;          /* fp32[n] weights */
    float* p_out;
    const void* g;           /* gradient[n] of grad_dtype */
    const void* m;
    void* m_out;
    const void* v;
    void* v_out;
    const uint8_t* m_scales;
    uint8_t* m_scales_out;
    const uint8_t* v_scales;
    uint8_t* v_scales_out;
    void* copy;              /* the new weights rounded to copy_dtype, or NULL */
    int64_t n;
    int64_t index;           /* enters the random bits: the tensor's place in the model, below 2^32 */
} sp24_adamw_tensor;

/* A step of AdamW (decoupled weight decay) over `count` tensors; in fp32, t the step from 1 on:
 *   g' = grad_scale * g;  m = beta1 m + (1 - beta1) g';  v = beta2 v + (1 - beta2) g'^2;
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps).
 * The update takes m and v as computed; then they are stored. A weight whose p, g, m and v are zero stays zero, so pruned
 * weights whose gradient is masked stay pruned.
 *   grad_dtype: BF16, FP16 or FP32. state_dtype: SP24_FP32 or SP24_FP8 (8 bits). copy_dtype: BF16 or FP16 (copies may be NULL).
 *   8-bit states are rounded up or down at random, with the odds that keep m and v right on average (rounded to nearest
 *   they would lose nearly every change of v: it moves by 1 - beta2 of itself a step), except that a v above zero is
 *   stored as at least one unit. The random bits are a hash of seed, t, index and the element's position: equal
 *   arguments give equal bits.
 *   lr_dev (fp32) and step_dev (int64): NULL, or device scalars that replace lr and step, read when the kernels run (a
 *   captured graph then follows them); workspace: 16 bytes, 16-byte aligned, then required, else NULL.
 *   grad_scale: NULL, or a device fp32 (loss scaling, clipping by the global norm).
 *   0 <= beta < 1, eps from 2^-126 on (its reciprocal is an fp32 number), lr and weight_decay finite and >= 0, step >= 1. A v below 2^-126 may
 *   count as zero under the root, which then is off by less than 2^-63. 1 - lr weight_decay and lr / (1 - beta1^t) are held within
 *   fp32's finite numbers. n at most 2^34. One launch for every 32 tensors;
 *   `tensors` is host memory, read before the call returns. Tensors must not overlap one another. */
int sp24_adamw(const sp24_adamw_tensor* tensors, int64_t count, int grad_dtype, int state_dtype, int copy_dtype, double lr,
               const float* lr_dev, int64_t step, const int64_t* step_dev, double beta1, double beta2, double eps,
               double weight_decay, const float* grad_scale, uint64_t seed, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SP24_LAYER_H */
