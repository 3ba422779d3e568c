// Device helpers of the 8-bit floating-point kernels (gfx950 only): e4m3 codes, e8m0 scales, rows of 16- and
// 32-bit numbers, and reductions.
#pragma once
#include "sp24_device.h"

namespace sp24 {

enum { T_BF16 = 0, T_FP16 = 1, T_FP32 = 2 };
template <int DT> constexpr int type_bytes() { return DT == T_FP32 ? 4 : 2; }

// Eight consecutive elements as stored: 16 bytes (32 for fp32).
template <int DT>
struct Raw8 {
    u32x4 w[DT == T_FP32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const char* p) {
    Raw8<DT> r;
    r.w[0] = *reinterpret_cast<const u32x4*>(p);
    if constexpr (DT == T_FP32) r.w[1] = *reinterpret_cast<const u32x4*>(p + 16);
    return r;
}
// The same with the non-temporal hint, for rows that are read once.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8_once(const char* p) {
    Raw8<DT> r;
    r.w[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    if constexpr (DT == T_FP32) r.w[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 16));
    return r;
}
template <int DT>
__device__ __forceinline__ Raw8<DT> zero8() {
    Raw8<DT> r;
    r.w[0] = u32x4{0, 0, 0, 0};
    if constexpr (DT == T_FP32) r.w[1] = u32x4{0, 0, 0, 0};
    return r;
}
template <int DT>
__device__ __forceinline__ void store8(char* p, const Raw8<DT>& r) {
    *reinterpret_cast<u32x4*>(p) = r.w[0];
    if constexpr (DT == T_FP32) *reinterpret_cast<u32x4*>(p + 16) = r.w[1];
}
template <int DT>
__device__ __forceinline__ float elem(const Raw8<DT>& r, int e) {
    if constexpr (DT == T_FP32) return __uint_as_float(r.w[e >> 2][e & 3]);
    const uint32_t h = (r.w[0][e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
    if constexpr (DT == T_BF16) return bf16_to_f32(h);
    return f16_to_f32(h);
}
// Eight fp32 values rounded once (to nearest even) to the stored type.
template <int DT>
__device__ __forceinline__ Raw8<DT> pack8(const float (&v)[8]) {
    Raw8<DT> r;
    if constexpr (DT == T_FP32) {
#pragma unroll
        for (int e = 0; e < 8; e++) r.w[e >> 2][e & 3] = __float_as_uint(v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++) {
            if constexpr (DT == T_BF16) {
                r.w[0][e] = pack_bf16x2_rne(v[2 * e], v[2 * e + 1]);
            } else {
                const uint16_t lo = __builtin_bit_cast(uint16_t, (_Float16)v[2 * e]);
                const uint16_t hi = __builtin_bit_cast(uint16_t, (_Float16)v[2 * e + 1]);
                r.w[0][e] = (uint32_t)lo | ((uint32_t)hi << 16);
            }
        }
    }
    return r;
}

// The scale byte of a block whose largest magnitude has the fp32 bits `amax`: 448 = 1.75 * 2^8, so the exponent
// field less 8, and one more where the fraction passes 0.75 (adding 0x1FFFFF carries into the exponent exactly
// there). At least 0 (2^-127); 255 (NaN) when the block holds an infinity or a NaN, whose bits order above
// every finite number's.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const int s = (int)((amax + 0x1FFFFFu) >> 23) - 8;
    return amax >= 0x7F800000u ? 255u : (uint32_t)(s < 0 ? 0 : s);
}
// 2^(127 - s): what a value is multiplied by before it is rounded to a code (exact, s <= 247; a NaN block's codes
// are unspecified).
__device__ __forceinline__ float code_factor(uint32_t s) { return __uint_as_float((254u - s) << 23); }
// 2^(s - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t s) {
    const uint32_t b = s << 23;
    return __uint_as_float((b > 0x00400000u ? b : 0x00400000u) + (((s + 1) >> 8) << 22));
}

// Two fp32 values rounded once (to nearest even) to packed bf16 or fp16.
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (!F16) return pack_bf16x2_rne(lo, hi);
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) | ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16);
}

// Four fp32 values (magnitudes within 448) rounded to nearest even to e4m3, element t in byte t.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
    return (uint32_t)v;
}

// Largest of a value over each 16 consecutive lanes (one DPP row), in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
#define SP24_ROR_MAX(n)                                                                              \
    {                                                                                                \
        const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + n, 0xF, 0xF, false);   \
        v = o > v ? o : v;                                                                           \
    }
    SP24_ROR_MAX(8) SP24_ROR_MAX(4) SP24_ROR_MAX(2) SP24_ROR_MAX(1)
#undef SP24_ROR_MAX
    return v;
}

// Sum over the 64 lanes, the same bits in all of them (rotations inside the DPP rows of 16 add the same pairs in
// every lane; the four rows in a fixed order).
__device__ __forceinline__ float wave_sum(float v) {
#define SP24_ROR_ADD(n) v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + n, 0xF, 0xF, false));
    SP24_ROR_ADD(8) SP24_ROR_ADD(4) SP24_ROR_ADD(2) SP24_ROR_ADD(1)
#undef SP24_ROR_ADD
    const int b = __float_as_int(v);
    const float r0 = __int_as_float(__builtin_amdgcn_readlane(b, 0)), r1 = __int_as_float(__builtin_amdgcn_readlane(b, 16));
    const float r2 = __int_as_float(__builtin_amdgcn_readlane(b, 32)), r3 = __int_as_float(__builtin_amdgcn_readlane(b, 48));
    return (r0 + r1) + (r2 + r3);
}

}  // namespace sp24
