// Gradient of the weight of a Linear layer from the 8-bit copy of its input: dW[m, k] = sum over tokens n of
// dY[n, m] x[n, k], dY in bf16, x in e4m3 codes with a power-of-two scale for each 128 channels of a token.
//
// A code times its scale is exactly a bf16 number (4 significant bits), so the product runs on the bf16 matrix
// cores (v_mfma_f32_16x16x32_bf16) with exact products and fp32 sums; the conversion is one instruction for two
// codes (v_cvt_scalef32_pk_bf16_fp8), done once an element while a tile is staged. Both operands have the summed
// index n as their slow axis; ds_read_b64_tr_b16 transposes them on the way from LDS to registers.
//
// Workgroup tile: 128 (k) x 128 (m), four waves of 64 x 64, 32 tokens a stage. LDS rows (one token) are 256 bytes in 8
// units of 32 bytes, unit u of row n at u ^ (2 (n & 3) + ((n >> 3) & 1)): the 16 rows of a transposing read
// (8 q + {0..3} for q = 0..3, 32 bytes each) then fall in 8 distinct units, two rows in each.
// A is x (rows k) and B is dY (columns m): an accumulator holds four consecutive k of one m, one 2:4 group, so a
// group's mask is one nibble and a store is 16 bytes (8 for bf16).
//
// Where the weight has too few tiles for the chip, the tokens are split over grid.z; each part writes fp32 sums to
// the workspace, and a second kernel adds the parts in order.
#include "fp8_device.h"
#include "sp24_launch.h"
#include "grad_weight_fp8.h"

namespace sp24 {
namespace {

constexpr int BT = 128, BN = 32;

struct Args {
    const char* dY;
    const uint8_t *X, *xs, *meta;
    char* out;
    int64_t N, M, K, lddy, ldx, lds, ldw;
    int64_t per;  // tokens of a part, a multiple of BN
    int64_t part_stride;
};

__device__ __forceinline__ int swz(int n) { return 2 * (n & 3) + ((n >> 3) & 1); }

// Four consecutive k of row m of the result.
template <bool F32>
__device__ __forceinline__ void store4(char* out, int64_t ldw, int64_t m, int64_t k, f32x4 v, const uint8_t* meta,
                                       int64_t tiles) {
    if (meta) v = masked(v, meta, m, k, tiles);
    if constexpr (F32) *reinterpret_cast<f32x4*>(out + (m * ldw + k) * 4) = v;
    else *reinterpret_cast<u32x2*>(out + (m * ldw + k) * 2) = u32x2{pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3])};
}

struct Staged {
    u32x4 x, y[2];
    uint32_t s;
};

template <bool F32>
__global__ __launch_bounds__(256) void grad_weight_kernel(Args a) {
    __shared__ __attribute__((aligned(16))) char sx[2][BN * 256];
    __shared__ __attribute__((aligned(16))) char sy[2][BN * 256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, q = lane >> 4;
    const int64_t k0 = (int64_t)blockIdx.x * BT, m0 = (int64_t)blockIdx.y * BT;
    const int64_t n_lo = (int64_t)blockIdx.z * a.per, n_hi = n_lo + a.per < a.N ? n_lo + a.per : a.N;
    const int wk = (wave >> 1) * 64, wm = (wave & 1) * 64;

    // x: thread t takes 16 codes (unit t % 8) of token t / 8; dY: 8 elements (unit t % 16) of tokens t / 16 and +16
    auto load = [&](int64_t n0) {
        Staged g;
        const int64_t n = n0 + (tid >> 3), k = k0 + 16 * (tid & 7);
        const bool ok = n < n_hi && k < a.K;
        g.x = ok ? *reinterpret_cast<const u32x4*>(a.X + n * a.ldx + k) : u32x4{0, 0, 0, 0};
        g.s = ok ? a.xs[n * a.lds + blockIdx.x] : 127u;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int64_t ny = n0 + (tid >> 4) + 16 * h, m = m0 + 8 * (tid & 15);
            const char* p = a.dY + (ny * a.lddy + m) * 2;
            u32x4 v = u32x4{0, 0, 0, 0};
            if (ny < n_hi && m + 7 < a.M) {
                v = *reinterpret_cast<const u32x4*>(p);
            } else if (ny < n_hi) {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (m + e < a.M) v[e >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
            }
            g.y[h] = v;
        }
        return g;
    };
    auto store = [&](const Staged& g, int buf) {
        const int n = tid >> 3, u = tid & 7;
        const float s = scale_value(g.s);
        u32x4 w[2];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            w[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(g.x[i], s, false));
            w[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(g.x[i], s, true));
        }
        char* const px = sx[buf] + n * 256 + ((u ^ swz(n)) << 5);
        *reinterpret_cast<u32x4*>(px) = w[0];
        *reinterpret_cast<u32x4*>(px + 16) = w[1];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int ny = (tid >> 4) + 16 * h, uy = (tid & 15) >> 1;
            *reinterpret_cast<u32x4*>(sy[buf] + ny * 256 + ((uy ^ swz(ny)) << 5) + 16 * (tid & 1)) = g.y[h];
        }
    };
    // fragment of 16 columns at c: lane (r, q) gets tokens 8 q .. 8 q + 7 of column c + r
    const int row = 8 * q + (r >> 2), roff = row * 256 + 8 * (r & 3), rs = swz(row);
    auto frag = [&](const char* base, int c) {
        typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
        const char* p = base + roff + (((c >> 4) ^ rs) << 5);
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p));
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 4 * 256));
        typedef short i16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(bf16x8, i16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    };

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    int buf = 0;
    if (n_lo < n_hi) {
        store(load(n_lo), 0);
        __syncthreads();
        for (int64_t n0 = n_lo; n0 < n_hi; n0 += BN, buf ^= 1) {
            const bool more = n0 + BN < n_hi;
            Staged g;
            if (more) g = load(n0 + BN);
            bf16x8 fx[4], fy[4];
#pragma unroll
            for (int i = 0; i < 4; i++) fx[i] = frag(sx[buf], wk + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; j++) fy[j] = frag(sy[buf], wm + 16 * j);
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[i], fy[j], acc[i][j], 0, 0, 0);
            if (more) store(g, buf ^ 1);
            __syncthreads();
        }
    }
    const int64_t tiles = (a.K + 127) / 128;
    char* const out = a.out + blockIdx.z * a.part_stride;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int64_t k = k0 + wk + 16 * i + 4 * q, m = m0 + wm + 16 * j + r;
            if (k < a.K && m < a.M) store4<F32>(out, a.ldw, m, k, acc[i][j], a.meta, tiles);
        }
}

// dW = the parts' sums in order; one thread for four columns.
template <bool F32>
__global__ __launch_bounds__(256) void add_parts_kernel(const float* __restrict__ part, int parts, int64_t M, int64_t K,
                                                        const uint8_t* __restrict__ meta, char* __restrict__ out,
                                                        int64_t ldw) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per_row = K / 4;
    if (i >= M * per_row) return;
    const int64_t m = i / per_row, k = 4 * (i - m * per_row);
    f32x4 v = *reinterpret_cast<const f32x4*>(part + m * K + k);
    for (int p = 1; p < parts; p++) v += *reinterpret_cast<const f32x4*>(part + (p * M + m) * K + k);
    store4<F32>(out, ldw, m, k, v, meta, (K + 127) / 128);
}

}  // namespace

// Parts that the tokens are split into: as many as still give the chip no more than two rounds of tiles, and at
// least 256 tokens a part.
int grad_weight_parts(int64_t M, int64_t K, int64_t N) {
    const int64_t tiles = ((M + BT - 1) / BT) * ((K + BT - 1) / BT);
    const int64_t want = 512 / tiles, most = N / 256;
    const int64_t p = want < most ? want : most;
    return (int)(p < 1 ? 1 : p);
}

hipError_t launch_grad_weight(const Fp8GradArgs& g, hipStream_t s) {
    if (((g.M + 255) / 256) * ((g.K + 255) / 256) >= 200) return launch_grad_weight_tiled(g, s);
    const int parts = grad_weight_parts(g.M, g.K, g.N);
    Args a;
    a.dY = static_cast<const char*>(g.dY); a.X = g.X; a.xs = g.xs;
    a.N = g.N; a.M = g.M; a.K = g.K; a.lddy = g.lddy; a.ldx = g.ldx; a.lds = g.lds;
    const int64_t per = (g.N + parts - 1) / parts;
    a.per = (per + BN - 1) / BN * BN;
    const dim3 grid((unsigned)((g.K + BT - 1) / BT), (unsigned)((g.M + BT - 1) / BT), (unsigned)parts);
    if (parts == 1) {
        a.meta = g.meta; a.out = static_cast<char*>(g.dW); a.ldw = g.ldw; a.part_stride = 0;
        if (g.out_fp32) hipLaunchKernelGGL((grad_weight_kernel<true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((grad_weight_kernel<false>), grid, dim3(256), 0, s, a);
        return hipGetLastError();
    }
    a.meta = nullptr; a.out = static_cast<char*>(g.workspace); a.ldw = g.K; a.part_stride = g.M * g.K * 4;
    hipLaunchKernelGGL((grad_weight_kernel<true>), grid, dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 add((unsigned)((g.M * (g.K / 4) + 255) / 256));
    if (g.out_fp32)
        hipLaunchKernelGGL((add_parts_kernel<true>), add, dim3(256), 0, s, static_cast<const float*>(g.workspace), parts,
                           g.M, g.K, g.meta, static_cast<char*>(g.dW), g.ldw);
    else
        hipLaunchKernelGGL((add_parts_kernel<false>), add, dim3(256), 0, s, static_cast<const float*>(g.workspace), parts,
                           g.M, g.K, g.meta, static_cast<char*>(g.dW), g.ldw);
    return hipGetLastError();
}

}  // namespace sp24
