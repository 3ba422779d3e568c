// Sparse x dense product in 8-bit floating point for a few tokens, with a scale for each block of 128.
//
// With N small the product streams the compressed weight (0.625 bytes a dense weight) from HBM once, and the
// codes of X stay in L2. A workgroup owns R consecutive 16-row blocks and 16 NF tokens; its S waves split the K
// tiles (128 dense columns, one block of scales, one v_smfmac_f32_16x16x128_fp8_fp8 a fragment) into contiguous
// ranges. A wave requests U tiles' operands at a time before their products: per lane and row block the 16-byte run
// of its slot in the value tile and its 32-bit index, per fragment the two 16-byte runs of its token's row that are
// the operand's halves (k0 + 16 q and k0 + 64 + 16 q), and the scales of the tile. A tile's product starts from
// zero; then acc = fma(product, 2^(x scale + w scale), acc), the power of two formed once a fragment and tile. (A
// NaN scale of the weight is noted beside the loop and put into the sums after it: as a factor in the loop, 11008 x 4096 at
// N = 16 took 12.5 us against 9.2.)
//
// Reads go through buffer descriptors: row blocks past M, tokens past N, runs past K (inside a row as well: what
// follows there may be a NaN code, which a zero weight would not cancel) and tiles past a wave's range read zeros.
// The waves' sums are added through LDS in wave order.
//
// The weight's bytes bound it where there are enough of them: 28672 x 8192 at one token 28.9 us, 5.1 TB/s, 11008 x 4096 8.3
// us, 3.4 TB/s; a 10 MB weight (4096 x 4096, 4.7 us; 4.0 where the weight is in the Infinity Cache) is a launch and two
// trips to memory.
#pragma once
#include "epilogue.h"

namespace sp24 {
namespace {

constexpr int KT = 128;
constexpr uint32_t OOR = 0x80000000u;  // a byte offset past every record count

struct Args {
    const uint8_t *values, *meta, *ws, *X, *xs;
    void* Y;
    int64_t M, K, N, ldx, lds, ldy;
    int y_vec;
    Epilogue epi;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
    const int64_t n = bytes <= 0 ? 0 : (bytes > 0x7FFFFFFFll ? 0x7FFFFFFFll : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)n, 0x00020000);
}

template <int NF, int R, int U, int S, bool F16, bool EPI>
__global__ __launch_bounds__(64 * S) void gemm_fp8_fewtok_kernel(Args a) {
    __shared__ f32x4 red[(EPI ? S : S - 1) * R * NF * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int64_t nb = (a.M + 15) / 16, b0 = (int64_t)blockIdx.x * R, n0 = (int64_t)blockIdx.y * 16 * NF;
    const int T = (int)((a.K + KT - 1) / KT);
    Epilogue epi;
    if constexpr (EPI) epi = read_early(a.epi);
    const int64_t blocks = nb - b0 < R ? nb - b0 : R;
    const int64_t tokens = a.N - n0 < 16 * NF ? a.N - n0 : 16 * NF;
    const __amdgpu_buffer_rsrc_t rA = rsrc(a.values + b0 * T * 1024, blocks * T * 1024);
    const __amdgpu_buffer_rsrc_t rM = rsrc(a.meta + b0 * T * 256, blocks * T * 256);
    const __amdgpu_buffer_rsrc_t rX = rsrc(a.X + n0 * a.ldx, (tokens - 1) * a.ldx + a.K);
    // eight row blocks share a row of weight scales; where R does not divide 8 the workgroup's last ones may be of the next
    constexpr bool TWO = 8 % R != 0;
    const uint8_t* ws = a.ws + (b0 >> 3) * T;
    const uint8_t* ws2 = a.ws + ((b0 + blocks - 1) >> 3) * T;
    uint32_t xo[NF];
    const uint8_t* xs[NF];  // tokens past N take the last one's scales: their products are zeros, and not stored
#pragma unroll
    for (int f = 0; f < NF; f++) {
        const int64_t n = 16 * f + r;
        xo[f] = n < tokens ? (uint32_t)(n * a.ldx + 16 * q) : OOR;
        xs[f] = a.xs + (n0 + (n < tokens ? n : tokens - 1)) * a.lds;
    }
    const int per = (T + S - 1) / S, t0 = wave * per, t1 = t0 + per < T ? t0 + per : T;

    f32x4 acc[R][NF];
#pragma unroll
    for (int i = 0; i < R; i++)
#pragma unroll
        for (int f = 0; f < NF; f++) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};

    uint32_t most = 0, most2 = 0;  // the largest weight scales: 255 makes the sums NaN after the loop

#pragma unroll 1
    for (int t = t0; t < t1; t += U) {
        i32x4 av[U][R];
        int iv[U][R];
        i32x8 bv[U][NF];
        uint32_t sx[U][NF], sw[U], sw2[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const bool in = t + u < t1;
            const int tc = in ? t + u : t;  // scales of tiles past the range: any valid one (their products are zeros)
            const int k0 = (t + u) * KT + 16 * q;
            sw[u] = ws[tc];
            if constexpr (TWO) sw2[u] = ws2[tc];
#pragma unroll
            for (int f = 0; f < NF; f++) sx[u][f] = xs[f][tc];
#pragma unroll
            for (int i = 0; i < R; i++) {
                const uint32_t ta = in ? (uint32_t)((i * T + t + u) * 1024 + 16 * lane) : OOR;
                const uint32_t tm = in ? (uint32_t)((i * T + t + u) * 256 + 4 * lane) : OOR;
                av[u][i] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rA, (int)ta, 0, 0));
                iv[u][i] = (int)__builtin_amdgcn_raw_buffer_load_b32(rM, (int)tm, 0, 0);
            }
#pragma unroll
            for (int f = 0; f < NF; f++) {
                const uint32_t o = xo[f] + (uint32_t)((t + u) * KT);
                const uint32_t o0 = in && k0 < a.K ? o : OOR, o1 = in && k0 + 64 < a.K ? o + 64u : OOR;
                const i32x4 lo = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rX, (int)o0, 0, 0));
                const i32x4 hi = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rX, (int)o1, 0, 0));
                bv[u][f] = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            most = max(most, sw[u]);
            if constexpr (TWO) most2 = max(most2, sw2[u]);
#pragma unroll
            for (int f = 0; f < NF; f++) {
                const float x = scale_value(sx[u][f]), s1 = __builtin_amdgcn_ldexpf(x, (int)sw[u] - 127);
                const float s2 = TWO ? __builtin_amdgcn_ldexpf(x, (int)sw2[u] - 127) : s1;
#pragma unroll
                for (int i = 0; i < R; i++) {
                    const float s = TWO && ((b0 + i) >> 3) != (b0 >> 3) ? s2 : s1;
                    const f32x4 p = __builtin_amdgcn_smfmac_f32_16x16x128_fp8_fp8(av[u][i], bv[u][f], f32x4{0.f, 0.f, 0.f, 0.f}, iv[u][i], 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[i][f][e] = fmaf(p[e], s, acc[i][f][e]);
                }
            }
        }
    }
    if (max(most, most2) == 255u) {
#pragma unroll
        for (int i = 0; i < R; i++)
            if ((TWO && ((b0 + i) >> 3) != (b0 >> 3) ? most2 : most) == 255u)
#pragma unroll
                for (int f = 0; f < NF; f++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[i][f][e] = __uint_as_float(0x7FC00000u);
    }
    if constexpr (EPI) {
        // Every wave finishes its share of the fragments: the activations' code, met for the first time here, is then fetched and
        // run once a wave and not once a fragment (11008 x 4096 at N = 37 with bias and SiLU 15.8 us with the first wave alone).
        constexpr int OT = F16 ? T_FP16 : T_BF16, COUNT = R * NF, MINE = (COUNT + S - 1) / S;
        const Places at = places(epi, static_cast<char*>(a.Y), a.ldy, false, 0);
        raw4<OT> res[MINE] = {};
        f32x4 bias[MINE] = {};
#pragma unroll
        for (int k = 0; k < MINE; k++) {  // on their way during the last sums
            const int j = wave + S * k;
            const int64_t m = 16 * (b0 + j / NF) + 4 * q, n = n0 + 16 * (j % NF) + r;
            const int in = a.M - m >= 4 ? 4 : a.M - m <= 0 ? 0 : (int)(a.M - m);
            if (j >= COUNT || n >= a.N || in == 0) continue;
            bias[k] = bias4(epi, m, in);
            res[k] = residual4<OT>(at, n, m, in);
        }
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int f = 0; f < NF; f++) red[((wave * R + i) * NF + f) * 64 + lane] = acc[i][f];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < MINE; k++) {
            const int j = wave + S * k;
            const int64_t m = 16 * (b0 + j / NF) + 4 * q, n = n0 + 16 * (j % NF) + r;
            const int in = a.M - m >= 4 ? 4 : a.M - m <= 0 ? 0 : (int)(a.M - m);
            if (j >= COUNT || n >= a.N || in == 0) continue;
            f32x4 y = red[j * 64 + lane];
#pragma unroll 1
            for (int w = 1; w < S; w++) y += red[(w * COUNT + j) * 64 + lane];
            finish4<OT>(epi, at, y, bias[k], res[k], n, m, in);
        }
        return;
    }
    if (wave > 0) {
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int f = 0; f < NF; f++) red[(((wave - 1) * R + i) * NF + f) * 64 + lane] = acc[i][f];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll 1
    for (int w = 1; w < S; w++)
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int f = 0; f < NF; f++) acc[i][f] += red[(((w - 1) * R + i) * NF + f) * 64 + lane];

    // lane (q, r): output channels 16 b + 4 q .. +3 of token 16 f + r
#pragma unroll
    for (int i = 0; i < R; i++) {
        const int64_t m0 = 16 * (b0 + i) + 4 * q;
        if (m0 >= a.M) continue;
#pragma unroll
        for (int f = 0; f < NF; f++) {
            const int64_t n = n0 + 16 * f + r;
            if (n >= a.N) continue;
            const f32x4 y = acc[i][f];
            uint16_t* const p = static_cast<uint16_t*>(a.Y) + n * a.ldy + m0;
            const u32x2 w = u32x2{pack16<F16>(y[0], y[1]), pack16<F16>(y[2], y[3])};
            if (a.y_vec && m0 + 3 < a.M) {
                *reinterpret_cast<u32x2*>(p) = w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (m0 + e < a.M) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
}

template <int NF, int R, int U, int S, bool EPI>
hipError_t launch(const Fp8GemmArgs& g, hipStream_t s) {
    Args a;
    a.values = g.values; a.meta = g.meta; a.ws = g.ws; a.X = g.X; a.xs = g.xs; a.Y = g.Y;
    a.M = g.M; a.K = g.K; a.N = g.N; a.ldx = g.ldx; a.lds = g.lds; a.ldy = g.ldy;
    a.y_vec = g.ldy % 4 == 0;  // Y is 16-byte aligned
    a.epi = g.epi;
    const dim3 grid((unsigned)(((g.M + 15) / 16 + R - 1) / R), (unsigned)((g.N + 16 * NF - 1) / (16 * NF)));
    if (g.out_fp16)
        hipLaunchKernelGGL((gemm_fp8_fewtok_kernel<NF, R, U, S, true, EPI>), grid, dim3(64 * S), 0, s, a);
    else
        hipLaunchKernelGGL((gemm_fp8_fewtok_kernel<NF, R, U, S, false, EPI>), grid, dim3(64 * S), 0, s, a);
    return hipGetLastError();
}

}  // namespace

// Row blocks a workgroup (R), tiles a request (U) and waves (S), measured on MI355X with weights rotated beyond the
// Infinity Cache (us):
//  R is the least of 1, 2 and 3 that leaves at most one workgroup a compute unit, and 4 (8 with one fragment) beyond; the
//  fewer, the more often each workgroup's X is read again, and at most 8 tokens are too few for that to count:
//  one fragment: 4096 x 4096 (256 row blocks) at N = 1 / 8 / 16 4.8 / 5.1 / 6.1 with R = 1; 8192 x 8192 (512) at N = 1 / 8
//    9.8 / 11.9 with R = 1, 11.8 / 11.7 with 2, at N = 16 12.1 with R = 2 against 15.5 with 1; 11008 x 4096 (688) at N = 1 / 8
//    8.2 / 8.8 with R = 2 against 8.1 / 9.5 with 1, at N = 16 9.3 with R = 3 against 10.9 with 4; 14336 x 4096 (896) at N =
//    16 11.9 with R = 4 against 12.8 with 3; 28672 x 8192 (1792) at N = 1 / 8 28.6 / 30.0 with R = 2 against 27.7 / 35.9 with
//    1, at N = 16 31.5 with R = 8 against 36.5 with 4;
//  two (N = 32): 4096 x 4096 8.8 with R = 1 against 9.5 with 2, 8192 x 8192 16.5 with 2 against 25.8 with 1, 11008 x 4096
//    12.5 with 3 and with 4 alike, 28672 x 8192 37.0 with 4 against 46.5 with 3;
//  three (N = 40; 37 the last two): 4096 x 4096 10.3 with R = 1 against 11.5 with 2, 8192 x 8192 19.8 with 2 against 32.2
//    with 1, 11008 x 4096 13.2 with 3 against 14.3 with 4, 28672 x 8192 41.2 with 4 against 51.4 with 3;
//  four, and groups of 64 tokens: 4096 x 4096 at N = 64 14.5 with R = 1 against 17.9 with 4, at N = 100 15.3 with 2, at N =
//    190 18.2 with 4 against 26.9 with 3 (258 workgroups); 11008 x 4096 at N = 64 17.3 with 3 against 19.1 with 4.
// The groups stream the weight once each, from L2 after the first; the tiled kernel reads it once but fills the chip
// only with many tiles. Up to 2.25 workgroups of 64 x 64 a compute unit this one is the faster (4096 x 4096 at N = 512, 2:
// 29.6 against 34.3 us; 11008 x 4096 at N = 200, 2.7: 41.7 against 35.4; 28672 x 8192 at N = 64, 1.75: 56.3 against 64.9, at
// N = 100, 3.5: 88.4 against 70.3).
inline bool few_tokens(const Fp8GemmArgs& g) {
    const int64_t nb = (g.M + 15) / 16, groups = (g.N + 63) / 64;
    return g.N <= 64 || 4 * ((nb + 3) / 4) * groups <= 9 * device_cus();
}

template <bool EPI>
hipError_t launch_fewtok(const Fp8GemmArgs& g, hipStream_t s) {
    const int64_t nb = (g.M + 15) / 16, groups = (g.N + 63) / 64, cus = device_cus();
    int per = 1;  // the least R, up to 5, with at most one workgroup a compute unit
    while (per < 5 && (nb + per - 1) / per * groups > cus) per++;
    if (g.N <= 8) return per <= 2 ? launch<1, 1, 4, 4, EPI>(g, s) : launch<1, 2, 2, 4, EPI>(g, s);
    if (g.N <= 16) {
        if (per <= 1) return launch<1, 1, 4, 4, EPI>(g, s);
        if (per <= 2) return launch<1, 2, 2, 4, EPI>(g, s);
        if (per <= 3) return launch<1, 3, 2, 4, EPI>(g, s);
        return per <= 4 ? launch<1, 4, 4, 8, EPI>(g, s) : launch<1, 8, 2, 8, EPI>(g, s);
    }
    if (g.N <= 32) {
        if (per <= 1) return launch<2, 1, 2, 4, EPI>(g, s);
        if (per <= 2) return launch<2, 2, 2, 4, EPI>(g, s);
        return per <= 3 ? launch<2, 3, 1, 8, EPI>(g, s) : launch<2, 4, 1, 8, EPI>(g, s);
    }
    if (g.N <= 48) {
        if (per <= 1) return launch<3, 1, 2, 4, EPI>(g, s);
        if (per <= 2) return launch<3, 2, 2, 8, EPI>(g, s);
        return per <= 3 ? launch<3, 3, 2, 4, EPI>(g, s) : launch<3, 4, 2, 4, EPI>(g, s);
    }
    if (per <= 1) return launch<4, 1, 2, 4, EPI>(g, s);
    if (per <= 2) return launch<4, 2, 2, 4, EPI>(g, s);
    return per <= 3 ? launch<4, 3, 2, 4, EPI>(g, s) : launch<4, 4, 2, 4, EPI>(g, s);
}

}  // namespace sp24
