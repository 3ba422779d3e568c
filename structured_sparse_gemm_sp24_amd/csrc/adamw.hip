// AdamW over many tensors in one launch, moments in fp32 or in 8 bits.
//
// A workgroup takes 2048 elements of one tensor, eight a thread, which finds its tensor by counting first workgroups in the
// launch's arguments (32 tensors of them fit). Everything of an element is read at once, and nothing else of it is needed: the 16
// lanes that hold a block of 128 find its scales by exchanging maxima, so 8-bit states take one pass as well.
// HBM bounds it: 28 bytes an element with 32-bit states and 16 (and four for each 128) with 8-bit ones, gradients and copies in 16
// bits. Three projections of 11008 x 4096 and their vectors (135 million elements) 726 us, two of 28672 x 8192 in 8 bits (470 million)
// 1429 us, both 5.2 TB/s, as a large copy reaches. 16 small tensors take 3.2 us (4.7 with 8 bits): the launch and one trip to memory.
#include "adamw.h"
#include "fp8_device.h"

#include <cmath>

namespace sp24 {
namespace {

// 32 bits stirred: two rounds of a shift and a product with an odd constant (2^32 over the golden ratio, the fraction of
// the square root of 2).
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x9E3779B9u;
    x = (x ^ (x >> 15)) * 0x6A09E667u;
    return x ^ (x >> 16);
}

// x as fp32, at most the largest finite one: an infinite rate would make NaN of a weight that has nothing to change.
__host__ __device__ inline float finite(double x) {
    constexpr double MOST = 3.4028234663852886e+38;
    return (float)(x > MOST ? MOST : x < -MOST ? -MOST : x);
}

__host__ __device__ inline AdamScalars scalars_of(const AdamSchedule& h, double lr, int64_t step) {
    AdamScalars a;
    a.decay = finite(1.0 - lr * h.decay);
    a.rate = finite(lr / (1.0 - pow(h.beta1, (double)step)));
    a.root = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)step)));
    a.key = mix(mix(mix((uint32_t)h.seed) ^ (uint32_t)(h.seed >> 32)) ^ (uint32_t)step);
    return a;
}

__global__ void adam_scalars_kernel(AdamSchedule h, AdamScalars* out) {
    *out = scalars_of(h, h.lr_dev ? (double)*h.lr_dev : h.lr, h.step_dev ? *h.step_dev : h.step);
}

// Eight elements of a thread; `in` of them exist.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_in(const char* p, int in) {
    if (in == 8) return load8_once<DT>(p);
    Raw8<DT> r = zero8<DT>();
#pragma unroll
    for (int e = 0; e < 7; e++)
        if (e < in) {
            if constexpr (DT == T_FP32) r.w[e >> 2][e & 3] = reinterpret_cast<const uint32_t*>(p)[e];
            else r.w[0][e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
        }
    return r;
}
template <int DT>
__device__ __forceinline__ void store_in(char* p, const Raw8<DT>& r, int in) {
    if (in == 8) return store8<DT>(p, r);
#pragma unroll
    for (int e = 0; e < 7; e++)
        if (e < in) {
            if constexpr (DT == T_FP32) reinterpret_cast<uint32_t*>(p)[e] = r.w[e >> 2][e & 3];
            else reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(r.w[0][e >> 1] >> (16 * (e & 1)));
        }
}
__device__ __forceinline__ u32x2 load_bytes(const char* p, int in) {
    if (in == 8) return __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    u32x2 r = {0, 0};
#pragma unroll
    for (int e = 0; e < 7; e++)
        if (e < in) r[e >> 2] |= (uint32_t) reinterpret_cast<const uint8_t*>(p)[e] << (8 * (e & 3));
    return r;
}
__device__ __forceinline__ void store_bytes(char* p, const u32x2& r, int in) {
    if (in == 8) {
        *reinterpret_cast<u32x2*>(p) = r;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; e++)
        if (e < in) reinterpret_cast<uint8_t*>(p)[e] = (uint8_t)(r[e >> 2] >> (8 * (e & 3)));
}

__device__ __forceinline__ uint32_t byte_of(const u32x2& r, int e) { return (r[e >> 2] >> (8 * (e & 3))) & 0xFFu; }

// First moment as e4m3: |m| in units below 448, up by 16 random bits of the 20 that are cut off, so that the code is right
// on average. Below the least normal number codes count 2^-9.
__device__ __forceinline__ uint32_t first_code(float m, float unit, uint32_t r16) {
#pragma clang fp contract(off)
    const float x = fabsf(m) * unit;
    const uint32_t r20 = r16 << 4;
    const uint32_t small = ((uint32_t)(int)(x * 0x1p29f) + r20) >> 20, big = ((__float_as_uint(x) + r20) >> 20) - 960u;
    return ((x < 0x1p-6f ? small : big) & 0x7Fu) | ((__float_as_uint(m) >> 24) & 0x80u);
}

// Second moment: c = floor(sqrt(x)) or c + 1, up where 16 random bits are below (x - c^2) / (2 c + 1), which keeps c^2 right on
// average; at least 1 unless v is zero. The hardware's root is one unit in the last place off, so the floor is put right.
__device__ __forceinline__ uint32_t second_code(float v, float unit2, uint32_t r16) {
#pragma clang fp contract(off)
    const float x = v * unit2;
    float c = floorf(__builtin_amdgcn_sqrtf(x));
    c = c * c > x ? c - 1.0f : (c + 1.0f) * (c + 1.0f) <= x ? c + 1.0f : c;
    const float odds = (x - c * c) * 65536.0f;
    const uint32_t code = (uint32_t)(int)c + ((float)r16 * (2.0f * c + 1.0f) < odds ? 1u : 0u);
    return code == 0u && v > 0.0f ? 1u : code;
}

template <int GT, bool BITS8, int CT>
__global__ __launch_bounds__(256) void adamw_kernel(AdamArgs a) {
#pragma clang fp contract(off)
    const int lane = threadIdx.x & 63;
    // the tensor whose workgroups this one belongs to
    const uint32_t f = lane < a.count ? a.first[lane] : 0xFFFFFFFFu;
    const int at = __builtin_popcountll(__builtin_amdgcn_ballot_w64(f <= blockIdx.x)) - 1;
    const AdamTensor& t = a.t[at];
    const int64_t i0 = (int64_t)(blockIdx.x - a.first[at]) * ADAM_CHUNK + 8 * threadIdx.x;
    const int64_t left = t.n - i0;
    const int in = left >= 8 ? 8 : left <= 0 ? 0 : (int)left;
    const AdamScalars now = a.later ? *a.later : a.now;
    const float scale = a.grad_scale ? *a.grad_scale : 1.0f;

    const Raw8<T_FP32> p = load_in<T_FP32>(reinterpret_cast<const char*>(t.p + i0), in);
    const Raw8<GT> g = load_in<GT>(t.g + i0 * type_bytes<GT>(), in);
    float m[8], v[8], w[8];
    if constexpr (BITS8) {
        const int64_t b = i0 >> 7;
        const u32x2 mc = load_bytes(t.m + i0, in), vc = load_bytes(t.v + i0, in);
        const uint32_t s1 = in ? t.ms[b] : 0u, s2 = in ? t.vs[b] : 0u;
        const float u1 = scale_value(s1);
        const float u2 = s2 == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((2u * (s2 < 64u ? 64u : s2) - 127u) << 23);  // 4^(s - 127)
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const float c = (float)byte_of(vc, e);
            const uint32_t code = byte_of(mc, e);
            m[e] = __builtin_amdgcn_cvt_f32_fp8((int)code, 0) * u1;
            v[e] = (c * c) * u2;
        }
    } else {
        const Raw8<T_FP32> mr = load_in<T_FP32>(t.m + i0 * 4, in), vr = load_in<T_FP32>(t.v + i0 * 4, in);
#pragma unroll
        for (int e = 0; e < 8; e++) m[e] = elem<T_FP32>(mr, e), v[e] = elem<T_FP32>(vr, e);
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const float ge = elem<GT>(g, e) * scale;
        m[e] = m[e] * a.b1 + ge * a.c1;
        v[e] = v[e] * a.b2 + (ge * ge) * a.c2;
        const float den = __builtin_amdgcn_sqrtf(v[e]) * now.root + a.eps;
        w[e] = elem<T_FP32>(p, e) * now.decay - now.rate * m[e] * __builtin_amdgcn_rcpf(den);
    }
    if (in) store_in<T_FP32>(reinterpret_cast<char*>(t.p_out + i0), pack8<T_FP32>(w), in);
    if constexpr (CT != T_FP32) {
        if (t.copy && in) store_in<CT>(t.copy + i0 * 2, pack8<CT>(w), in);
    }
    if constexpr (BITS8) {
        uint32_t big1 = 0, big2 = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const uint32_t b1 = e < in ? __float_as_uint(m[e]) & 0x7FFFFFFFu : 0u, b2 = e < in ? __float_as_uint(v[e]) & 0x7FFFFFFFu : 0u;
            big1 = max(big1, b1), big2 = max(big2, b2);
        }
        big1 = max16(big1), big2 = max16(big2);  // the 16 lanes of a block
        const uint32_t s1 = scale_byte(big1);
        // the least even k with the largest v within 255^2 2^k (0x477E0100 is 255^2), at least -126
        const int k = ((int)(big2 - 0x477E0100u) + 0x7FFFFF) >> 23;
        const int h = (k + 1) >> 1;
        const uint32_t s2 = big2 >= 0x7F800000u ? 255u : (uint32_t)((h < -63 ? -63 : h) + 127);
        const float unit1 = code_factor(s1), unit2 = __uint_as_float((uint32_t)(127 - 2 * ((int)s2 - 127)) << 23);
        const uint32_t key = mix(now.key + t.index * 0x9E3779B9u) + (uint32_t)(i0 >> 32) * 0x9E3779B9u;
        u32x2 mc = {0, 0}, vc = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const uint32_t r = mix((uint32_t)(i0 + e) * 0xBB67AE85u + key);
            mc[e >> 2] |= first_code(m[e], unit1, r & 0xFFFFu) << (8 * (e & 3));
            vc[e >> 2] |= (second_code(v[e], unit2, r >> 16) & 0xFFu) << (8 * (e & 3));
        }
        if (in) {
            store_bytes(t.m_out + i0, mc, in);
            store_bytes(t.v_out + i0, vc, in);
            if ((threadIdx.x & 15) == 0) t.ms_out[i0 >> 7] = (uint8_t)s1, t.vs_out[i0 >> 7] = (uint8_t)s2;
        }
    } else if (in) {
        store_in<T_FP32>(t.m_out + i0 * 4, pack8<T_FP32>(m), in);
        store_in<T_FP32>(t.v_out + i0 * 4, pack8<T_FP32>(v), in);
    }
}

template <int GT, bool BITS8>
hipError_t launch_copy(const AdamArgs& a, int copy, unsigned blocks, hipStream_t s) {
    const dim3 grid(blocks), block(256);
    if (copy == T_BF16) hipLaunchKernelGGL((adamw_kernel<GT, BITS8, T_BF16>), grid, block, 0, s, a);
    else if (copy == T_FP16) hipLaunchKernelGGL((adamw_kernel<GT, BITS8, T_FP16>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((adamw_kernel<GT, BITS8, T_FP32>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

AdamScalars adam_scalars(const AdamSchedule& h) { return scalars_of(h, h.lr, h.step); }

hipError_t launch_adam_scalars(const AdamSchedule& h, AdamScalars* out, hipStream_t s) {
    hipLaunchKernelGGL(adam_scalars_kernel, dim3(1), dim3(1), 0, s, h, out);
    return hipGetLastError();
}

hipError_t launch_adamw(const AdamArgs& a, int grad, bool bits8, int copy, unsigned blocks, hipStream_t s) {
    switch (grad) {
    case T_BF16: return bits8 ? launch_copy<T_BF16, true>(a, copy, blocks, s) : launch_copy<T_BF16, false>(a, copy, blocks, s);
    case T_FP16: return bits8 ? launch_copy<T_FP16, true>(a, copy, blocks, s) : launch_copy<T_FP16, false>(a, copy, blocks, s);
    default: return bits8 ? launch_copy<T_FP32, true>(a, copy, blocks, s) : launch_copy<T_FP32, false>(a, copy, blocks, s);
    }
}

}  // namespace sp24
