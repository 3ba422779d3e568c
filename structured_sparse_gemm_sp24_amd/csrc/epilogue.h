// Fused epilogue of the 2:4 products (gfx950 only), and the derivatives of its activations:
//   z = acc + bias[m],  Z = round(z),  y = act(z) + R,  Y = round(y),  every step in fp32.
#pragma once
#include "fp8_device.h"
#include "sp24_launch.h"

namespace sp24 {

enum { ACT_NONE = 0, ACT_GELU = 1, ACT_RELU = 2, ACT_SILU = 3 };  // the sp24_activation numbers
constexpr int NO_EPILOGUE = -1;  // in place of an activation: the plain product

// erfc(a / sqrt 2) / 2 for 0 <= a <= 20 and e^{-a^2 / 2}, as in gelu_f32 (Abramowitz & Stegun 7.1.26).
__device__ __forceinline__ float half_erfc(float a, float& gauss) {
#pragma clang fp contract(off)
    constexpr float P = (float)(as7126::P * 0.70710678118654752), C = (float)(-0.5 * 1.4426950408889634);
    const float pa = a * P;
    const float s = pa * __builtin_amdgcn_rcpf(pa + 1.0f);
    float q = as7126::half_b(5);
    q = fmaf(s, q, as7126::half_b(4));
    q = fmaf(s, q, as7126::half_b(3));
    q = fmaf(s, q, as7126::half_b(2));
    q = fmaf(s, q, as7126::half_b(1));
    q = fmaf(s, q, as7126::half_b(0));
    gauss = __builtin_amdgcn_exp2f((a * C) * a);
    return q * gauss;
}
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}
// |z| up to 20, where e^{-z^2 / 2} is zero in fp32: infinities then give no product of infinity and zero. NaN stays.
__device__ __forceinline__ float within20(float z) { return __builtin_elementwise_minimum(fabsf(z), 20.0f); }
constexpr float LARGEST = 3.402823466e+38f;

template <int ACT>
__device__ __forceinline__ float act_f32(float z) {
    if constexpr (ACT == ACT_RELU) return __builtin_elementwise_maximum(z, 0.0f);  // NaN stays
    if constexpr (ACT == ACT_GELU) {
        float gauss;
        const float a = within20(z);
        return fmaf(-a, half_erfc(a, gauss), __builtin_elementwise_maximum(z, 0.0f));
    }
    if constexpr (ACT == ACT_SILU) return __builtin_elementwise_maximum(z, -LARGEST) * sigmoid(z);
    return z;
}
__device__ __forceinline__ float act_any(float z, int act) {
    return act == ACT_GELU ? act_f32<ACT_GELU>(z) : act == ACT_RELU ? act_f32<ACT_RELU>(z) : act == ACT_SILU ? act_f32<ACT_SILU>(z) : z;
}

// dy act'(z). GELU'(z) = Phi(z) + z phi(z); SiLU'(z) = s + z s (1 - s) with s = 1 / (1 + e^-z); ReLU chooses, so an
// infinite dy is lost where z <= 0.
template <int ACT>
__device__ __forceinline__ float act_back(float dy, float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? dy : 0.0f;
    if constexpr (ACT == ACT_GELU) {
        float gauss;
        const float a = within20(z), r = half_erfc(a, gauss);
        return dy * fmaf(copysignf(a, z) * 0.3989422804014327f, gauss, z > 0.0f ? 1.0f - r : r);
    }
    if constexpr (ACT == ACT_SILU) {
        const float s = sigmoid(z), zf = __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -LARGEST), LARGEST);
        return dy * fmaf(zf * s, 1.0f - s, s);
    }
    return dy;
}

// ---------------------------------------------------------------- four consecutive outputs of a row
template <int OT> struct Four { typedef u32x2 raw; };
template <> struct Four<T_FP32> { typedef u32x4 raw; };
template <int OT> using raw4 = typename Four<OT>::raw;
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));

template <int OT>
__device__ __forceinline__ f32x4 widen4(const raw4<OT>& w) {
    if constexpr (OT == T_FP32) return f32x4{__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3])};
    else if constexpr (OT == T_BF16)
        return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u), __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xFFFF0000u)};
    else return f32x4{f16_to_f32(w[0] & 0xFFFFu), f16_to_f32(w[0] >> 16), f16_to_f32(w[1] & 0xFFFFu), f16_to_f32(w[1] >> 16)};
}
template <int OT>
__device__ __forceinline__ raw4<OT> narrow4(const f32x4& y) {
    if constexpr (OT == T_FP32) return u32x4{__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])};
    else return u32x2{pack16<OT == T_FP16>(y[0], y[1]), pack16<OT == T_FP16>(y[2], y[3])};
}
// Even: the address is a multiple of 8 (16-bit types) or 16 bytes and the line is not needed again here; else any element's.
template <int OT, bool EVEN>
__device__ __forceinline__ raw4<OT> read4(const char* p) {
    if constexpr (EVEN) return __builtin_nontemporal_load(reinterpret_cast<const raw4<OT>*>(p));
    else if constexpr (OT == T_FP32) return *reinterpret_cast<const u32x4_at4*>(p);
    else return *reinterpret_cast<const u32x2_at2*>(p);
}
template <int OT, bool EVEN>
__device__ __forceinline__ void write4(char* p, const raw4<OT>& w) {
    if constexpr (EVEN) __builtin_nontemporal_store(w, reinterpret_cast<raw4<OT>*>(p));
    else if constexpr (OT == T_FP32) *reinterpret_cast<u32x4_at4*>(p) = w;
    else *reinterpret_cast<u32x2_at2*>(p) = w;
}
// The first `in` of the four.
template <int OT>
__device__ __forceinline__ raw4<OT> read_in(const char* p, int in) {
    if (in == 4) return read4<OT, false>(p);
    raw4<OT> w = {};
#pragma unroll
    for (int t = 0; t < 3; t++)
        if (t < in) {
            if constexpr (OT == T_FP32) w[t] = reinterpret_cast<const uint32_t*>(p)[t];
            else w[t >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[t] << (16 * (t & 1));
        }
    return w;
}
template <int OT>
__device__ __forceinline__ void write_in(char* p, const raw4<OT>& w, int in) {
    if (in == 4) return write4<OT, false>(p, w);
#pragma unroll
    for (int t = 0; t < 3; t++)
        if (t < in) {
            if constexpr (OT == T_FP32) reinterpret_cast<uint32_t*>(p)[t] = w[t];
            else reinterpret_cast<uint16_t*>(p)[t] = (uint16_t)(w[t >> 1] >> (16 * (t & 1)));
        }
}

// The outputs' places of one batch entry: rows of `length` elements, `rows` of them (tokens or, feature-major, channels).
struct Places {
    char *Y, *Z;
    const char* R;
    int64_t ldy, ldz, ldr, rows, length;
};

// Places of batch entry `entry` (its Y given), for the kernels that need neither rows nor length.
__device__ __forceinline__ Places places(const Epilogue& e, char* y, int64_t ldy, bool fp32, int64_t entry) {
    const int64_t es = fp32 ? 4 : 2;
    return {y, e.Z ? static_cast<char*>(e.Z) + entry * e.sz * es : nullptr, e.R ? static_cast<const char*>(e.R) + entry * e.sr * es : nullptr,
            ldy, e.ldz, e.ldr, 0, 0};
}

// The epilogue of the batch entries from b0 on.
inline Epilogue entries_from(Epilogue e, int64_t b0, bool fp32) {
    if (e.R) e.R = static_cast<const char*>(e.R) + b0 * e.sr * (fp32 ? 4 : 2);
    if (e.Z) e.Z = static_cast<char*>(e.Z) + b0 * e.sz * (fp32 ? 4 : 2);
    return e;
}

// The epilogue and the output of a kernel whose only argument has a member epi, Y, ldy, M and N, read here and not at the
// kernel's start: kept in scalar registers through the main loop they would push out others.
template <typename Args>
__device__ __forceinline__ const __attribute__((address_space(4))) Args* late_args() {
    auto k = (const __attribute__((address_space(4))) Args*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(k));
    return k;
}

// One output, the activation chosen at run time: the kernels for few tokens.
__device__ __forceinline__ void finish1(const Epilogue& e, const Places& p, int type, float acc, float bias, int64_t row, int64_t col) {
    const float z = e.bias ? acc + bias : acc;
    float y = act_any(z, e.act);
    const int64_t oy = row * p.ldy + col, oz = row * p.ldz + col, orr = row * p.ldr + col;
    if (type == T_FP32) {
        if (p.R) y += reinterpret_cast<const float*>(p.R)[orr];
        if (p.Z) reinterpret_cast<float*>(p.Z)[oz] = z;
        reinterpret_cast<float*>(p.Y)[oy] = y;
    } else {
        if (p.R) {
            const uint32_t r = reinterpret_cast<const uint16_t*>(p.R)[orr];
            y += type == T_BF16 ? bf16_to_f32(r) : f16_to_f32(r);
        }
        if (p.Z) reinterpret_cast<uint16_t*>(p.Z)[oz] = (uint16_t)(type == T_BF16 ? pack16<false>(z, z) : pack16<true>(z, z));
        reinterpret_cast<uint16_t*>(p.Y)[oy] = (uint16_t)(type == T_BF16 ? pack16<false>(y, y) : pack16<true>(y, y));
    }
}

// f(0) .. f(N - 1), each with its index as a constant (as a loop the compiler may refuse to unroll, and with it to keep
// accumulators in registers).
template <int N>
struct Index {
    static constexpr int value = N;
    __device__ constexpr operator int() const { return N; }
};
template <int N, typename F>
__device__ __forceinline__ void each(const F& f) {
    if constexpr (N > 0) {
        each<N - 1>(f);
        f(Index<N - 1>());
    }
}

// A wave's place in one of Y, Z and R, four rows of it at a time. FULL: the wave's block lies inside, and every row on 8 or 16
// bytes: a uniform address, 32-bit offsets of the lanes, and the lines are not needed again here. Otherwise an address a lane,
// at any element.
template <int OT, bool FULL>
struct Rows {
    static constexpr int ES = OT == T_FP32 ? 4 : 2;
    uint64_t at;
    uint32_t lane;
    int64_t pitch;  // bytes

    __device__ __forceinline__ Rows(const void* base, int64_t ld, int64_t row0, int64_t col0, int row, int col) {
        pitch = ld * ES;
        at = reinterpret_cast<uint64_t>(base) + (uint64_t)(row0 * pitch + col0 * ES);
        lane = (uint32_t)(row * pitch + col * ES);
        if constexpr (!FULL) at += (uint64_t)(row * pitch + col * ES);
    }
    __device__ __forceinline__ char* place(int slot, int cols) const {
        return reinterpret_cast<char*>(at + (uint64_t)(slot * pitch + cols * ES)) + (FULL ? lane : 0u);
    }
    // Sixteen rows on. The address is kept from the optimizer, which would else compute all of them ahead and run out of registers.
    __device__ __forceinline__ void advance() {
        at += (uint64_t)(16 * pitch);
        if constexpr (FULL) asm volatile("" : "+s"(at));
        else asm volatile("" : "+v"(at));
    }
    __device__ __forceinline__ raw4<OT> read(int slot, int cols, int in) const {
        if constexpr (FULL) return read4<OT, true>(place(slot, cols));
        else return read_in<OT>(place(slot, cols), in);
    }
    __device__ __forceinline__ void write(int slot, int cols, const f32x4& v, int in) const {
        if constexpr (FULL) write4<OT, true>(place(slot, cols), narrow4<OT>(v));
        else write_in<OT>(place(slot, cols), narrow4<OT>(v), in);
    }
};

// Epilogue of a wave's 128 channels x 16 FNT tokens from accumulators acc(i, j) whose lane (q, r) holds channels 16 i + 4 q
// .. +3 of token 16 j + r. The transposes of the plain product's stores run on the fp32 sums, so that bias, activation and
// residual all work on the four consecutive outputs of a row that a lane stores: token-major four channels of a token,
// feature-major four tokens of a channel.
template <bool TM, int OT, int ACT, bool FULL, int FNT, typename Acc>
__device__ __forceinline__ void store_fused(const Acc& acc, const float* bias, const Places& p, int64_t mw, int64_t nw, int lane) {
    constexpr int OUTER = TM ? FNT : 8, INNER = TM ? 2 : FNT / 4;  // groups of 16 rows, of 64 columns
    const int q = lane >> 4, r = lane & 15, x = r & 3, c = r >> 2;
    const int64_t row0 = TM ? nw : mw, col0 = TM ? mw : nw;
    const int row = TM ? 4 * c : 4 * q, col = TM ? 16 * x + 4 * q : 16 * x + 4 * c;
    Rows<OT, FULL> y(p.Y, p.ldy, row0, col0, row, col), z(p.Z, p.ldz, row0, col0, row, col), res(p.R, p.ldr, row0, col0, row, col);
    int64_t rows_left = p.rows - row0 - row, cols_left = p.length - col0 - col;  // from the lane's place on

    f32x4 tb[TM ? 2 : 1] = {};  // token-major: the lane's channels
    if constexpr (TM) {
        if (bias) {
#pragma unroll
            for (int g = 0; g < 2; g++)
#pragma unroll
                for (int t = 0; t < 4; t++)
                    if (FULL || cols_left > 64 * g + t) tb[g][t] = bias[col0 + col + 64 * g + t];
        }
    }
    each<OUTER>([&](auto o) __attribute__((always_inline)) {
        f32x4 fb = {0.f, 0.f, 0.f, 0.f};  // feature-major: the slots' channels
        if constexpr (!TM) {
            if (bias) {
#pragma unroll
                for (int s = 0; s < 4; s++)
                    if (FULL || rows_left > s) fb[s] = bias[row0 + row + 16 * o + s];
            }
        }
        each<INNER>([&](auto g) __attribute__((always_inline)) {
            int in[4];
            raw4<OT> rv[4] = {};
            if constexpr (!FULL) {
                const int64_t left = cols_left - 64 * g;
                const int cols = left >= 4 ? 4 : left <= 0 ? 0 : (int)left;
#pragma unroll
                for (int s = 0; s < 4; s++) in[s] = rows_left > s ? cols : 0;
            }
            if (p.R) {
#pragma unroll
                for (int s = 0; s < 4; s++) rv[s] = res.read(s, 64 * g, in[s]);
            }
            uint32_t v[4][4];
#pragma unroll
            for (int f = 0; f < 4; f++) {
                const f32x4 a = TM ? acc(4 * g + f, o) : acc(o, 4 * g + f);
#pragma unroll
                for (int t = 0; t < 4; t++) v[f][t] = __float_as_uint(a[t]);
                if constexpr (!TM) quad_transpose(v[f], x);
            }
            slot_transpose4<4>(v, x);
#pragma unroll
            for (int s = 0; s < 4; s++) {
                f32x4 zv, yv;
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    zv[t] = __uint_as_float(v[s][t]) + (TM ? tb[TM ? g.value : 0][t] : fb[s]);
                    yv[t] = act_f32<ACT>(zv[t]);
                }
                if (p.Z) z.write(s, 64 * g, zv, in[s]);
                if (p.R) yv += widen4<OT>(rv[s]);
                y.write(s, 64 * g, yv, in[s]);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        y.advance(), z.advance(), res.advance();
        if constexpr (!FULL) rows_left -= 16;
    });
}

}  // namespace sp24
