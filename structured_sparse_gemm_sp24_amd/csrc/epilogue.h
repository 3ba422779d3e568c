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
// Memory of the operands as such: an address made from a number would else be of any kind, and its access a slower one.
#define SP24_GLOBAL __attribute__((address_space(1)))
typedef SP24_GLOBAL char global_char;
template <typename T>
__device__ __forceinline__ SP24_GLOBAL T* global_at(const char* p) { return (SP24_GLOBAL T*)p; }
template <typename T>
__device__ __forceinline__ SP24_GLOBAL T* global_at(const global_char* p) { return (SP24_GLOBAL T*)p; }

// EVEN: the address is a multiple of 8 (16-bit types) or 16 bytes and the line is not needed again here; else any element's.
template <int OT, bool EVEN, typename P>
__device__ __forceinline__ raw4<OT> read4(P p) {
    if constexpr (EVEN) return __builtin_nontemporal_load(global_at<const raw4<OT>>(p));
    else if constexpr (OT == T_FP32) return *global_at<const u32x4_at4>(p);
    else return *global_at<const u32x2_at2>(p);
}
template <int OT, bool EVEN, typename P>
__device__ __forceinline__ void write4(P p, const raw4<OT>& w) {
    if constexpr (EVEN) __builtin_nontemporal_store(w, global_at<raw4<OT>>(p));
    else if constexpr (OT == T_FP32) *global_at<u32x4_at4>(p) = w;
    else *global_at<u32x2_at2>(p) = w;
}
// The first `in` of the four.
template <int OT, typename P>
__device__ __forceinline__ raw4<OT> read_in(P p, int in) {
    if (in == 4) return read4<OT, false>(p);
    raw4<OT> w = {};
#pragma unroll
    for (int t = 0; t < 3; t++)
        if (t < in) {
            if constexpr (OT == T_FP32) w[t] = global_at<const uint32_t>(p)[t];
            else w[t >> 1] |= (uint32_t)global_at<const uint16_t>(p)[t] << (16 * (t & 1));
        }
    return w;
}
template <int OT, typename P>
__device__ __forceinline__ void write_in(P p, const raw4<OT>& w, int in) {
    if (in == 4) return write4<OT, false>(p, w);
#pragma unroll
    for (int t = 0; t < 3; t++)
        if (t < in) {
            if constexpr (OT == T_FP32) global_at<uint32_t>(p)[t] = w[t];
            else global_at<uint16_t>(p)[t] = (uint16_t)(w[t >> 1] >> (16 * (t & 1)));
        }
}

// The outputs' places of one batch entry: rows of `length` elements, `rows` of them (tokens or, feature-major, channels).
struct Places {
    char *Y, *Z;
    const char* R;
    int64_t ldy, ldz, ldr, rows, length;
};

// What a fused epilogue needs, in the arguments of a tiled kernel. Through the main loop a wave keeps it in one vector
// register, a word a lane: in scalar registers it would push out others, and read again from the kernel's arguments, which
// may lie in the host's memory, each tile would wait for it.
struct Outputs {
    char *Y, *Z;
    const char* R;
    const float* bias;
    int64_t ldy, ldz, ldr, sy, sz, sr, M, N;  // strides of batch entries in elements
    int64_t rows;  // one of these
};
// Rows of Y, Z and R: 16 of one take 2^31 bytes or more; every one on 8 (16-bit types) or 16 bytes, or on 64 where the outputs are large
// (below), and then the whole of Y takes 64 MB or more; else ODD. A residual is usually what was written last: a small one is read through the caches, which may
// still hold it (768 x 768 over 6304 tokens 16.4 us against 18.0, 512 x 128 over 32 x 784 23.8 against 31.3, buffers in turn), a large
// one past them (11008 x 4096 over 4096 tokens 187 against 195).
// Outputs go out past the caches. Where rows share 64-byte lines the caches join the pieces instead, once Y takes 8 MB with a Z beside it
// or 32 MB alone (past the caches / through them: 11000 x 4096 over 4096 tokens with bias 202 / 187, with GELU and Z 266 / 217, 1000 x 768
// over 20000 38.7 / 32.7, over 6304 with all 30.8 / 28.7; below 17.3 / 17.9, 512 x 128 over 32 x 784 with residual 24.4 / 25.8).
enum { WIDE, ODD, EVEN, EVEN_LARGE };
constexpr int OUTPUT_WORDS = sizeof(Outputs) / 4;
static_assert(OUTPUT_WORDS <= 64, "a word a lane");

__device__ __forceinline__ uint32_t keep_outputs(const Outputs& o, int lane) {
    uint32_t w = reinterpret_cast<const uint32_t*>(&o)[lane < OUTPUT_WORDS ? lane : 0];
    asm volatile("" : "+v"(w));  // not read again
    return w;
}
__device__ __forceinline__ Outputs kept_outputs(uint32_t kept) {
    uint32_t w[OUTPUT_WORDS];
#pragma unroll
    for (int i = 0; i < OUTPUT_WORDS; i++) w[i] = (uint32_t)__builtin_amdgcn_readlane((int)kept, i);
    return __builtin_bit_cast(Outputs, w);
}
inline Outputs outputs_of(const Epilogue& e, void* Y, int64_t ldy, int64_t sy, int64_t M, int64_t N, int es, int64_t batch) {
    Outputs o{static_cast<char*>(Y), static_cast<char*>(e.Z), static_cast<const char*>(e.R), e.bias, ldy, e.ldz, e.ldr, sy, e.sz, e.sr, M, N, EVEN};
    const int64_t bytes = M * N * batch * es, unit = bytes >= ((int64_t)(e.Z ? 8 : 32) << 20) ? 64 : 4 * es;
    const auto look = [&](const void* p, int64_t ld, int64_t stride) {
        if (p && ((ld * es) % unit != 0 || (batch > 1 && (stride * es) % unit != 0)) && o.rows == EVEN) o.rows = ODD;
        if (p && ld * es * 16 >= ((int64_t)1 << 31)) o.rows = WIDE;
    };
    look(Y, ldy, sy);
    look(e.R, e.ldr, e.sr);
    look(e.Z, e.ldz, e.sz);
    if (o.rows == EVEN && bytes >= ((int64_t)64 << 20)) o.rows = EVEN_LARGE;
    return o;
}
template <bool TM>
__device__ __forceinline__ Places places_of(const Outputs& o, int64_t entry, int es) {
    return {o.Y + entry * o.sy * es, o.Z ? o.Z + entry * o.sz * es : nullptr, o.R ? o.R + entry * o.sr * es : nullptr,
            o.ldy, o.ldz, o.ldr, TM ? o.N : o.M, TM ? o.M : o.N};
}

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

// One output from z = acc + bias and its residual, the activation chosen at run time: the kernels for few tokens.
__device__ __forceinline__ float residual1(const Places& p, int type, int64_t row, int64_t col) {
    if (!p.R) return 0.f;
    const int64_t o = row * p.ldr + col;
    if (type == T_FP32) return reinterpret_cast<const float*>(p.R)[o];
    const uint32_t r = reinterpret_cast<const uint16_t*>(p.R)[o];
    return type == T_BF16 ? bf16_to_f32(r) : f16_to_f32(r);
}
__device__ __forceinline__ void finish1(int act, const Places& p, int type, float z, float r, int64_t row, int64_t col) {
    float y = act_any(z, act);
    if (p.R) y += r;
    const int64_t oy = row * p.ldy + col, oz = row * p.ldz + col;
    if (type == T_FP32) {
        if (p.Z) reinterpret_cast<float*>(p.Z)[oz] = z;
        reinterpret_cast<float*>(p.Y)[oy] = y;
    } else {
        if (p.Z) reinterpret_cast<uint16_t*>(p.Z)[oz] = (uint16_t)(type == T_BF16 ? pack16<false>(z, z) : pack16<true>(z, z));
        reinterpret_cast<uint16_t*>(p.Y)[oy] = (uint16_t)(type == T_BF16 ? pack16<false>(y, y) : pack16<true>(y, y));
    }
}

template <int ACT>
__device__ __forceinline__ f32x4 act4(f32x4 z) {
    return f32x4{act_f32<ACT>(z[0]), act_f32<ACT>(z[1]), act_f32<ACT>(z[2]), act_f32<ACT>(z[3])};
}
__device__ __forceinline__ f32x4 act_any4(f32x4 z, int act) {
    if (act == ACT_NONE) return z;
    return act == ACT_GELU ? act4<ACT_GELU>(z) : act == ACT_RELU ? act4<ACT_RELU>(z) : act4<ACT_SILU>(z);
}

// Four consecutive outputs of a row from column col on, `in` of them inside, the activation chosen at run time, with bias and
// residual that were requested before.
template <int OT>
__device__ __forceinline__ raw4<OT> residual4(const Places& p, int64_t row, int64_t col, int in) {
    if (!p.R) return raw4<OT>{};
    return read_in<OT>(p.R + (row * p.ldr + col) * (OT == T_FP32 ? 4 : 2), in);
}
__device__ __forceinline__ f32x4 bias4(const Epilogue& e, int64_t col, int in) {
    if (!e.bias) return f32x4{0.f, 0.f, 0.f, 0.f};
    return widen4<T_FP32>(read_in<T_FP32>(reinterpret_cast<const char*>(e.bias + col), in));
}
template <int OT>
__device__ __forceinline__ void finish4(const Epilogue& e, const Places& p, const f32x4& acc, const f32x4& b, const raw4<OT>& r, int64_t row,
                                        int64_t col, int in) {
    constexpr int ES = OT == T_FP32 ? 4 : 2;
    const f32x4 z = acc + b;
    f32x4 y = act_any4(z, e.act);
    if (p.R) y += widen4<OT>(r);
    if (p.Z) write_in<OT>(p.Z + (row * p.ldz + col) * ES, narrow4<OT>(z), in);
    write_in<OT>(p.Y + (row * p.ldy + col) * ES, narrow4<OT>(y), in);
}

// The epilogue's arguments read at the kernel's start: where the compiler would read them, at its end, they are a trip to the
// host's memory.
__device__ __forceinline__ Epilogue read_early(const Epilogue& a) {
    Epilogue e = a;
    asm volatile("" : "+s"(e.bias), "+s"(e.R), "+s"(e.Z), "+s"(e.ldr), "+s"(e.ldz), "+s"(e.sr), "+s"(e.sz), "+s"(e.act));
    return e;
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

// How a wave's block lies in Y: wholly inside; with rows past the end; with columns past it too (or rows so long that 32-bit
// offsets do not reach over 16 of them).
enum { WHOLE, SOME_ROWS, ANYHOW };

// A wave's place in one of Y, Z and R, four rows of it at a time: a uniform address and 32-bit offsets of the lanes, or ANYHOW an
// address a lane.
template <int OT, int BLOCK>
struct Rows {
    static constexpr int ES = OT == T_FP32 ? 4 : 2;
    uint64_t at;
    uint32_t lane;
    int64_t pitch;  // bytes

    __device__ __forceinline__ Rows(const void* base, int64_t ld, int64_t row0, int64_t col0, int row, int col) {
        pitch = ld * ES;
        at = reinterpret_cast<uint64_t>(base) + (uint64_t)(row0 * pitch + col0 * ES);
        lane = (uint32_t)(row * pitch + col * ES);
        if constexpr (BLOCK != ANYHOW) asm volatile("" : "+v"(lane));  // 32 bits, not widened and added ahead
        else at += (uint64_t)(row * pitch + col * ES);
    }
    __device__ __forceinline__ global_char* place(int slot, int cols) const {
        return (global_char*)(at + (uint64_t)(slot * pitch + cols * ES)) + (BLOCK != ANYHOW ? lane : 0u);
    }
    // Sixteen rows on. The address is kept from the optimizer, which would else compute all of them ahead and run out of registers.
    __device__ __forceinline__ void advance() {
        at += (uint64_t)(16 * pitch);
        if constexpr (BLOCK != ANYHOW) asm volatile("" : "+s"(at));
        else asm volatile("" : "+v"(at));
    }
    // in: how many of the four elements exist (SOME_ROWS: none or all). once: whole lines that are not needed again here go past
    // the caches; where rows share lines the caches join the pieces.
    __device__ __forceinline__ void read(raw4<OT> (&v)[4], int cols, bool once, const int (&in)[4]) const {
        if (BLOCK == WHOLE && once) {
            asm volatile("" ::: "memory");  // or the two branches become one, and the hint is lost
#pragma unroll
            for (int s = 0; s < 4; s++) v[s] = read4<OT, true>(place(s, cols));
            asm volatile("" ::: "memory");
            return;
        }
#pragma unroll
        for (int s = 0; s < 4; s++) {
            if constexpr (BLOCK == WHOLE) v[s] = read4<OT, false>(place(s, cols));
            else if constexpr (BLOCK == SOME_ROWS) v[s] = in[s] ? read4<OT, false>(place(s, cols)) : raw4<OT>{};
            else v[s] = read_in<OT>(place(s, cols), in[s]);
        }
    }
    __device__ __forceinline__ void write(const raw4<OT> (&v)[4], int cols, bool once, const int (&in)[4]) const {
        if constexpr (BLOCK == ANYHOW) {
#pragma unroll
            for (int s = 0; s < 4; s++) write_in<OT>(place(s, cols), v[s], in[s]);
        } else if constexpr (BLOCK == SOME_ROWS) {
#pragma unroll
            for (int s = 0; s < 4; s++)
                if (in[s]) write4<OT, false>(place(s, cols), v[s]);
        } else if (once) {
            asm volatile("" ::: "memory");  // as above
#pragma unroll
            for (int s = 0; s < 4; s++) write4<OT, true>(place(s, cols), v[s]);
            asm volatile("" ::: "memory");
        } else {
#pragma unroll
            for (int s = 0; s < 4; s++) write4<OT, false>(place(s, cols), v[s]);
        }
    }
};

// Two 4 x 4 transposes inside the lane quads (quad_transpose of sp24_device.h) in half the instructions: the exchange between
// two lanes and the choice of what to keep are one v_cndmask with a DPP source. Of two words on either side of the diagonal lane
// b of a quad keeps its own and takes the other from lane b ^ 2, then b ^ 1. The s_nop, and further on the order, keep two
// instructions between a register's write and its read through DPP. a and b must be results of vector instructions other
// than matrix and transcendental ones, whose waits the compiler does not put before an asm block.
__device__ __forceinline__ void quad_transpose2(uint32_t (&a)[4], uint32_t (&b)[4]) {
    uint32_t o[8], x[8];
    asm("s_nop 1\n\t"
        "s_mov_b64 vcc, %24\n\t"
        "v_cndmask_b32_dpp %8, %18, %16, vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %9, %19, %17, vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %12, %22, %20, vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %13, %23, %21, vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "s_not_b64 vcc, vcc\n\t"
        "v_cndmask_b32_dpp %10, %16, %18, vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %11, %17, %19, vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %14, %20, %22, vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %15, %21, %23, vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "s_mov_b64 vcc, %25\n\t"
        "v_cndmask_b32_dpp %0, %9, %8, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %2, %11, %10, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %4, %13, %12, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %6, %15, %14, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "s_not_b64 vcc, vcc\n\t"
        "v_cndmask_b32_dpp %1, %8, %9, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %3, %10, %11, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %5, %12, %13, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_cndmask_b32_dpp %7, %14, %15, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf"
        : "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]), "=&v"(o[4]), "=&v"(o[5]), "=&v"(o[6]), "=&v"(o[7]), "=&v"(x[0]), "=&v"(x[1]),
          "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "s"(0x3333333333333333ull),
          "s"(0x5555555555555555ull)
        : "vcc", "scc");
#pragma unroll
    for (int t = 0; t < 4; t++) a[t] = o[t], b[t] = o[4 + t];
}

// Epilogue of a wave's 128 channels x 16 FNT tokens from accumulators acc(i, j) whose lane (q, r) holds channels 16 i + 4 q
// .. +3 of token 16 j + r. The transposes of the plain product's stores run on the fp32 sums, so that activation and residual
// work on the four consecutive outputs of a row that a lane stores: token-major four channels of a token, feature-major four
// tokens of a channel. Groups of 16 rows x 64 columns, along a row first, so that token-major 256 consecutive bytes of a row go
// out together. The residual of a group is requested before the group in front of it is finished (HAS_R, 16-bit types, whole blocks; the other cases lack the
// registers, and whether there is a residual is then seen group by group). The bias is added as the sums lie; where they
// are results of vector instructions (VECTOR), after the transposes, which takes fewer registers.
template <bool TM, bool VECTOR, int OT, int ACT, int BLOCK, bool HAS_R, int FNT, typename Acc>
__device__ __forceinline__ void store_block(const Acc& acc, const float* bias, const Places& p, int64_t how, int64_t mw, int64_t nw, int lane) {
    constexpr int ROWS = TM ? FNT : 8, COLS = TM ? 2 : FNT / 4, GROUPS = ROWS * COLS;
    constexpr bool AHEAD = HAS_R && OT != T_FP32, LATE_BIAS = TM && VECTOR;
    static_assert(BLOCK == WHOLE || !HAS_R, "residuals are looked for group by group");
    const int q = lane >> 4, r = lane & 15, x = r & 3, c = r >> 2;
    const int64_t row0 = TM ? nw : mw, col0 = TM ? mw : nw;
    const int row = TM ? 4 * c : 4 * q, col = TM ? 16 * x + 4 * q : 16 * x + 4 * c;
    Rows<OT, BLOCK> y(p.Y, p.ldy, row0, col0, row, col), z(p.Z, p.ldz, row0, col0, row, col), res(p.R, p.ldr, row0, col0, row, col);
    const int64_t cols_left = p.length - col0 - col, rows_left = p.rows - row0 - row;  // from the lane's place on
    const auto inside = [&](int (&in)[4], int at_row, int at_col) __attribute__((always_inline)) {
        const int64_t left = BLOCK == ANYHOW ? cols_left - 64 * at_col : 4;
        const int cols = left >= 4 ? 4 : left <= 0 ? 0 : (int)left;
#pragma unroll
        for (int s = 0; s < 4; s++) in[s] = BLOCK == WHOLE || rows_left > 16 * at_row + s ? cols : 0;
    };
    const auto bias_at = [&](int64_t m) __attribute__((always_inline)) {
        const char* const at = reinterpret_cast<const char*>(bias + m);
        const int64_t left = (TM ? p.length : p.rows) - m;
        if constexpr (BLOCK == WHOLE || (BLOCK == SOME_ROWS && TM)) return widen4<T_FP32>(read4<T_FP32, false>(at));
        return widen4<T_FP32>(read_in<T_FP32>(at, left <= 0 ? 0 : left < 4 ? (int)left : 4));
    };
    constexpr int BIAS = !TM ? 1 : LATE_BIAS ? 2 : 8;  // of the row of fragments, of the lane's columns, of its fragments
    f32x4 b[BIAS] = {};
    if (TM && bias) {
#pragma unroll
        for (int f = 0; f < BIAS; f++) b[f] = bias_at(LATE_BIAS ? mw + 64 * f + col : mw + 16 * f + 4 * q);
    }
    raw4<OT> ahead[4];
    const auto request = [&](auto g) __attribute__((always_inline)) {
        int in[4];
        inside(in, g.value / COLS, g.value % COLS);
        if constexpr (g.value > 0 && g.value % COLS == 0) res.advance();
        res.read(ahead, 64 * (g.value % COLS), how == EVEN_LARGE, in);
    };
    if constexpr (AHEAD) request(Index<0>());
    each<GROUPS>([&](auto g) __attribute__((always_inline)) {
        constexpr int at_row = g.value / COLS, at_col = g.value % COLS;
        if constexpr (at_col == 0) {
            if constexpr (g.value > 0) y.advance(), z.advance();
            if (!TM && bias) b[0] = bias_at(mw + 16 * at_row + 4 * q);
        }
        raw4<OT> now[4];
        if constexpr (AHEAD) {
#pragma unroll
            for (int s = 0; s < 4; s++) now[s] = ahead[s];
            if constexpr (g.value + 1 < GROUPS) request(Index<g.value + 1>());
        }
        uint32_t v[4][4];  // v[t][f]: the lane's value t of fragment f, then of slot f
#pragma unroll
        for (int f = 0; f < 4; f++) {
            f32x4 a = TM ? acc(4 * at_col + f, at_row) : acc(at_row, 4 * at_col + f);
            if constexpr (!LATE_BIAS) a += b[TM ? 4 * at_col + f : 0];
#pragma unroll
            for (int t = 0; t < 4; t++) v[t][f] = __float_as_uint(a[t]);
        }
        if constexpr (!TM) {
            uint32_t w[4][4];  // w[f][t]
#pragma unroll
            for (int f = 0; f < 4; f++)
#pragma unroll
                for (int t = 0; t < 4; t++) w[f][t] = v[t][f];
            quad_transpose2(w[0], w[1]);
            quad_transpose2(w[2], w[3]);
#pragma unroll
            for (int f = 0; f < 4; f++)
#pragma unroll
                for (int t = 0; t < 4; t++) v[t][f] = w[f][t];
        }
        quad_transpose2(v[0], v[1]);
        quad_transpose2(v[2], v[3]);
        int in[4];
        raw4<OT> out[4];
        f32x4 zv[4], yv[4];
        inside(in, at_row, at_col);
#pragma unroll
        for (int s = 0; s < 4; s++) {
#pragma unroll
            for (int t = 0; t < 4; t++) zv[s][t] = __uint_as_float(v[t][s]);
            if constexpr (LATE_BIAS) zv[s] += b[at_col];
        }
        if (p.Z) {
#pragma unroll
            for (int s = 0; s < 4; s++) out[s] = narrow4<OT>(zv[s]);
            z.write(out, 64 * at_col, how >= EVEN, in);
        }
#pragma unroll
        for (int s = 0; s < 4; s++)
#pragma unroll
            for (int t = 0; t < 4; t++) yv[s][t] = act_f32<ACT>(zv[s][t]);
        if constexpr (AHEAD) {
#pragma unroll
            for (int s = 0; s < 4; s++) yv[s] += widen4<OT>(now[s]);
        } else if (HAS_R || (BLOCK != WHOLE && p.R)) {
            request(g);
#pragma unroll
            for (int s = 0; s < 4; s++) yv[s] += widen4<OT>(ahead[s]);
        }
#pragma unroll
        for (int s = 0; s < 4; s++) out[s] = narrow4<OT>(yv[s]);
        y.write(out, 64 * at_col, how >= EVEN, in);
        __builtin_amdgcn_sched_barrier(0);
    });
}

template <bool TM, bool VECTOR, int OT, int ACT, int FNT, typename Acc>
__device__ __forceinline__ void store_fused(const Acc& acc, const Outputs& o, const Places& p, int64_t mw, int64_t nw, int lane) {
    const bool rows = TM ? nw + 16 * FNT <= o.N : mw + 128 <= o.M, cols = (TM ? mw + 128 <= o.M : nw + 16 * FNT <= o.N) && o.rows != WIDE;
    if (!cols) store_block<TM, VECTOR, OT, ACT, ANYHOW, false, FNT>(acc, o.bias, p, o.rows, mw, nw, lane);
    else if (!rows) store_block<TM, VECTOR, OT, ACT, SOME_ROWS, false, FNT>(acc, o.bias, p, o.rows, mw, nw, lane);
    else if (p.R) store_block<TM, VECTOR, OT, ACT, WHOLE, true, FNT>(acc, o.bias, p, o.rows, mw, nw, lane);
    else store_block<TM, VECTOR, OT, ACT, WHOLE, false, FNT>(acc, o.bias, p, o.rows, mw, nw, lane);
}

}  // namespace sp24
