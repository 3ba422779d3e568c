// Gradient of the weight of a Linear layer from the 8-bit copy of its input: dW[m, k] = sum over tokens n of
// dY[n, m] x[n, k], dY in bf16, x in e4m3 codes with a power-of-two scale for each 128 channels of a token.
//
// A code times its scale is exactly a bf16 number (4 significant bits), so the product runs on the bf16 matrix
// cores (v_mfma_f32_16x16x32_bf16) with exact products and fp32 sums; the conversion is one instruction for two
// codes (v_cvt_scalef32_pk_bf16_fp8), done once an element while a tile is staged. Both operands have the summed
// index n as their slow axis; ds_read_b64_tr_b16 transposes them on the way from LDS to registers.
//
// Workgroup tile: 128 (k) x 128 (m), four waves of 64 x 64, 64 tokens a stage. LDS rows (one token) are 256 bytes in 8
// units of 32 bytes, unit u of row n at u ^ (2 (n & 3) + ((n >> 3) & 1)): the 16 rows of a transposing read
// (8 q + {0..3} for q = 0..3, 32 bytes each) then fall in 8 distinct units, two rows in each.
// A is x (rows k) and B is dY (columns m): an accumulator holds four consecutive k of one m, one 2:4 group, so a
// group's mask is one nibble and a store is 16 bytes (8 for bf16).
//
// Where the weight has too few tiles for the chip, the tokens are split; each part writes fp32 sums to
// the workspace, and a second kernel adds the parts in order.
//
// 768 x 768 over 6304 tokens (7 parts): 20.2 us and 4.2 for the sums. Its matrix instructions are 3.5 us; each of the 252
// workgroups reads its 24 KB a stage through its XCD's L2, 78 MB fetched in all for 14.5 MB of operands, at 3.9 TB/s,
// and writes 16.5 MB of partial sums. Stages of 32 tokens took 29.6 us in all against 27.9, 14 parts 30.8 us.
#include "fp8_device.h"
#include "sp24_launch.h"
#include "grad_weight_fp8.h"

namespace sp24 {
namespace {

constexpr int BT = 128, BN = 64;
constexpr int XH = BN / 32, YH = BN / 16;  // 16-byte loads of a thread in a stage: codes, dY

struct Args {
    const char* dY;
    const uint8_t *X, *xs, *meta;
    char* out;
    int64_t N, M, K, lddy, ldx, lds, ldw;
    int64_t per;  // tokens of a part, a multiple of 2 BN
    int64_t part_stride;
    int tiles, tilesK;
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

constexpr uint32_t OOR = 0x80000000u;  // a byte offset past every record count, also with a row's offset added
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes, bool any) {
    const int64_t n = !any ? 0 : (bytes > 0x7FFFFFF0ll ? 0x7FFFFFF0ll : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)n, 0x00020000);
}

struct Staged {
    u32x4 x[XH], y[YH];
    uint32_t s[XH];
};

template <bool F32>
__global__ __launch_bounds__(256) void grad_weight_kernel(Args a) {
    __shared__ __attribute__((aligned(16))) char sx[2][BN * 256];
    __shared__ __attribute__((aligned(16))) char sy[2][BN * 256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, q = lane >> 4;
    const int part = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int tk = tile % a.tilesK, tm = tile / a.tilesK;
    const int64_t k0 = (int64_t)tk * BT, m0 = (int64_t)tm * BT;
    const int64_t n_lo = (int64_t)part * a.per, n_hi = n_lo + a.per < a.N ? n_lo + a.per : a.N;
    const int wk = (wave >> 1) * 64, wm = (wave & 1) * 64;

    // x: thread t takes 16 codes (unit t % 8) of token t / 8; dY: 8 elements (unit t % 16) of tokens t / 16 and +16. Loads
    // through descriptors and without branches, so that the compiler can count what is in flight: units past K, tokens
    // past the part's end and elements past dY's end read zeros; elements past M inside a row feed sums that are not
    // stored.
    const bool xk = k0 + 16 * (tid & 7) < a.K;
    const uint32_t xo = xk ? (uint32_t)((tid >> 3) * (int)a.ldx + 16 * (tid & 7)) : OOR;
    const uint32_t so = xk ? (uint32_t)((tid >> 3) * (int)a.lds) : OOR;
    const uint32_t yo = m0 + 8 * (tid & 15) < a.M ? (uint32_t)(((tid >> 4) * (int)a.lddy + 8 * (tid & 15)) * 2) : OOR;
    auto load = [&](int64_t n0) {
        Staged g;
        const int64_t left = n_hi - 1 - n0;  // descriptors of no bytes from n_hi on
        const __amdgpu_buffer_rsrc_t rx = rsrc(a.X + n0 * a.ldx + k0, left * a.ldx + a.K - k0, left >= 0);
        const __amdgpu_buffer_rsrc_t rs = rsrc(a.xs + n0 * a.lds + tk, left * a.lds + 1, left >= 0);
        const __amdgpu_buffer_rsrc_t ry = rsrc(a.dY + (n0 * a.lddy + m0) * 2, ((left * a.lddy + a.M - m0) * 2 + 3) & ~(int64_t)3, left >= 0);
#pragma unroll
        for (int h = 0; h < XH; h++) {
            g.x[h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(xo + 32u * h * (uint32_t)a.ldx), 0, 0));
            g.s[h] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rs, (int)(so + 32u * h * (uint32_t)a.lds), 0, 0);
        }
#pragma unroll
        for (int h = 0; h < YH; h++)
            g.y[h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ry, (int)(yo + 32u * h * (uint32_t)a.lddy), 0, 0));
        return g;
    };
    auto store = [&](const Staged& g, int buf) {
#pragma unroll
        for (int h = 0; h < XH; h++) {
            const int n = (tid >> 3) + 32 * h, u = tid & 7;
            const float s = scale_value(g.s[h]);
            u32x4 w[2];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                w[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(g.x[h][i], s, false));
                w[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(g.x[h][i], s, true));
            }
            char* const px = sx[buf] + n * 256 + ((u ^ swz(n)) << 5);
            *reinterpret_cast<u32x4*>(px) = w[0];
            *reinterpret_cast<u32x4*>(px + 16) = w[1];
        }
#pragma unroll
        for (int h = 0; h < YH; h++) {
            const int ny = (tid >> 4) + 16 * h, uy = (tid & 15) >> 1;
            *reinterpret_cast<u32x4*>(sy[buf] + ny * 256 + ((uy ^ swz(ny)) << 5) + 16 * (tid & 1)) = g.y[h];
        }
    };
    // fragment of 16 columns at c in step t: lane (r, q) gets tokens 32 t + 8 q .. + 7 of column c + r
    const int row = 8 * q + (r >> 2), roff = row * 256 + 8 * (r & 3), rs = swz(row);
    auto frag = [&](const char* base, int c, int t) {
        typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
        const char* p = base + roff + t * (32 * 256) + (((c >> 4) ^ rs) << 5);
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

    // Stage n0 from buffer `buf`: `use` holds the next stage's operands, loaded a stage ago, `next` takes those of the one
    // after it. The two alternate without copies, which would wait for the loads just issued.
    auto step = [&](int64_t n0, int buf, const Staged& use, Staged& next) {
        next = load(n0 + 2 * BN);  // zeros from n_hi on
#pragma unroll
        for (int t = 0; t < BN / 32; t++) {
            bf16x8 fx[4], fy[4];
#pragma unroll
            for (int i = 0; i < 4; i++) fx[i] = frag(sx[buf], wk + 16 * i, t);
#pragma unroll
            for (int j = 0; j < 4; j++) fy[j] = frag(sy[buf], wm + 16 * j, t);
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[i], fy[j], acc[i][j], 0, 0, 0);
        }
        store(use, buf ^ 1);
        __syncthreads();
    };
    if (n_lo < n_hi) {
        Staged g0 = load(n_lo), g1 = load(n_lo + BN);
        store(g0, 0);
        __syncthreads();
        for (int64_t n0 = n_lo; n0 < n_hi; n0 += 2 * BN) {  // the last stage may be one of zeros
            step(n0, 0, g1, g0);
            step(n0 + BN, 1, g0, g1);
        }
    }
    const int64_t tiles = (a.K + 127) / 128;
    char* const out = a.out + part * a.part_stride;
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

// Parts that the tokens are split into: as many as keep the workgroups within one a compute unit of 256, at least
// 256 tokens a part, and none without tokens, a part being whole steps of 128 (768 x 768 over 6304 tokens, 36 tiles: 27.9 us with 7 parts, 30.8 with 14; 1024 x 4096 over 2048 tokens,
// 256 tiles: 37.7 in one part, 41.2 in two; 2048 x 1024 over 300 tokens: 15.6 in one part, 22.5 in two).
int grad_weight_parts(int64_t M, int64_t K, int64_t N) {
    const int64_t tiles = ((M + BT - 1) / BT) * ((K + BT - 1) / BT);
    const int64_t want = 256 / tiles, most = N / 256;
    const int64_t p = want < most ? want : most;
    if (p < 2) return 1;
    const int64_t steps = (N + 2 * BN - 1) / (2 * BN), per = (steps + p - 1) / p;  // whole steps a part
    return (int)((steps + per - 1) / per);
}

// The 256 x 256 kernel (one workgroup a compute unit) where its rounds of the chip are full enough: in one round, where the
// tiles of 128 x 128 would take more than one of their own (two workgroups a compute unit); in two, from two thirds full;
// always from three. Measured (us, 128 wide / 256 wide; tiles of 256 x 256): 2816 x 2816 over 8192 tokens (121) 160 / 202, 2048
// x 4096 over 4096 (128) 98 / 113, 768 x 11008 over 8192 (129) 232 / 202, 4096 x 2304 over 4096 (144) 134 / 115, 4096 x
// 4096 over 4096 (256) 165 / 122; 5120 x 4096 over 4096 (320) 199 / 220, 5632 x 4096 over 2048 (352) 131 / 127, 5120 x
// 5120 over 2048 (400) 151 / 127; 11008 x 4096 over 4096 (688) 427 / 334.
static bool grad_weight_takes_tiled(int64_t M, int64_t K) {
    const int64_t cus = device_cus(), big = ((M + 255) / 256) * ((K + 255) / 256);
    const int64_t small = ((M + BT - 1) / BT) * ((K + BT - 1) / BT), rounds = (big + cus - 1) / cus;
    if (rounds == 1) return small > 2 * cus;
    return 3 * big >= 2 * cus * rounds;
}

hipError_t launch_grad_weight(const Fp8GradArgs& g, hipStream_t s) {
    if (grad_weight_takes_tiled(g.M, g.K)) return launch_grad_weight_tiled(g, s);
    const int parts = grad_weight_parts(g.M, g.K, g.N);
    Args a;
    a.dY = static_cast<const char*>(g.dY); a.X = g.X; a.xs = g.xs;
    a.N = g.N; a.M = g.M; a.K = g.K; a.lddy = g.lddy; a.ldx = g.ldx; a.lds = g.lds;
    const int64_t per = (g.N + parts - 1) / parts;
    a.per = (per + 2 * BN - 1) / (2 * BN) * (2 * BN);
    a.tilesK = (int)((g.K + BT - 1) / BT);
    a.tiles = a.tilesK * (int)((g.M + BT - 1) / BT);
    const dim3 grid((unsigned)(a.tiles * parts));
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
