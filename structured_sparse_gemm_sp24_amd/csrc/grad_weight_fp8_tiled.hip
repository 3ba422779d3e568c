// Gradient of the weight from the 8-bit copy of the input, for weights with tiles enough for the chip (the formulas and
// the operands' layout are in grad_weight_fp8.hip): workgroup tile 256 (k) x 256 (m), eight waves of 128 x 64, two a
// SIMD, 8 x 4 fragments of v_mfma_f32_16x16x32_bf16 (128 sums a lane). While one wave of a SIMD converts codes, reads
// fragments or stores, the other's matrix instructions run: 11008 x 4096 over 4096 tokens 338 us (1.09 PFLOP/s) on one
// set of inputs, 357 to 365 us on three in turn; 8192^3 917 us (1.20), against 382 and 1037 us (on one set) with four waves
// of 128 x 128, which read a quarter less LDS; v_mfma_f32_32x32x16_bf16
// was slower. Matrix cores are busy 42 % of the cycles at 2.15 GHz; what bounds it is the conversion and LDS traffic beside them
// (every code is written to LDS as bf16 and read back transposed) and the last, part-full round of tiles.
//
// A stage is 64 tokens, two steps of 32. LDS holds two stages of x (bf16, 512 bytes a token) and dY; unit u of 32 bytes
// of token n is stored at u ^ (2 (n & 3) + ((n >> 3) & 1)), which keeps the transposing reads free of conflicts.
// While step t is multiplied, the fragments of step t + 1 are read. In the first step of stage s the codes of stage
// s + 1, loaded a stage before, are converted and written to the other buffer; the barrier between the steps
// publishes that buffer (its dY has landed by then) and frees this one, whose fragments are all in registers: into
// it go the loads of dY of stage s + 2, and the codes of stage s + 2 into registers.
#include "fp8_device.h"
#include "sp24_launch.h"
#include "grad_weight_fp8.h"

namespace sp24 {
namespace {

constexpr int BT = 256, BN = 64, WK = 128, WM = 64, FK = WK / 16, FM = WM / 16;
constexpr int HALF_BYTES = BN * BT * 2, STAGE_BYTES = 2 * HALF_BYTES;  // x, then dY
constexpr uint32_t OOR = 0x80000000u;
constexpr int GROUP = 8;

struct Args {
    const char* dY;
    const uint8_t *X, *xs, *meta;
    char* out;
    int64_t N, M, K, lddy, ldx, lds, ldw;
    int tilesK, tilesM, vec;
};

__device__ __forceinline__ i32x4 make_rsrc(const void* base, int64_t bytes) {
    const int64_t n = bytes <= 0 ? 0 : (bytes > 0x7FFFFFF0ll ? 0x7FFFFFF0ll : bytes);
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    r[1] = __builtin_amdgcn_readfirstlane((int)((b >> 32) & 0xFFFFu));
    r[2] = __builtin_amdgcn_readfirstlane((int)(uint32_t)n);
    r[3] = 0x00020000;
    return r;
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
    const int64_t n = bytes <= 0 ? 0 : (bytes > 0x7FFFFFF0ll ? 0x7FFFFFF0ll : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)n, 0x00020000);
}
__device__ __forceinline__ void dma16(uint32_t lds, uint32_t voff, const i32x4& r) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(r) : "memory");
}

__device__ __forceinline__ int swz(int n) { return 2 * (n & 3) + ((n >> 3) & 1); }

typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

// 16 columns of a step: lane (r, q) gets tokens 8 q .. 8 q + 7 of column r (p: the lane's place for these columns).
__device__ __forceinline__ bf16x8 frag(uint32_t p) {
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(const lds_char*)(size_t)p);
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(const lds_char*)(size_t)(p + 4 * 512));
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, i16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}

// A thread's codes of a stage: unit (16 codes) t % 16 of tokens t / 16 + 32 h, and their scales.
struct Codes {
    u32x4 x[2];
    uint32_t s[2];
};

template <bool F32>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void grad_weight_tiled_kernel(Args a) {
    __shared__ __attribute__((aligned(128))) char smem[2 * STAGE_BYTES];
    const uint32_t l0 = (uint32_t)(size_t)(lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, q = lane >> 4;

    // tile: workgroups of one XCD (p % 8) take neighbouring tiles, walked in groups of GROUP tile columns
    int L;
    {
        const int T = gridDim.x, p = blockIdx.x, x = p & 7, i = p >> 3, q8 = T >> 3, r8 = T & 7;
        L = x * q8 + (x < r8 ? x : r8) + i;
    }
    const int gsize = GROUP * a.tilesK, grp = L / gsize, first = grp * GROUP;
    const int gm = (a.tilesM - first) < GROUP ? (a.tilesM - first) : GROUP, in_g = L - grp * gsize;
    const int64_t m0 = (int64_t)(first + in_g % gm) * BT, k0 = (int64_t)(in_g / gm) * BT;
    const int wk = (wave >> 2) * WK, wm = (wave & 3) * WM;
    const int S = (int)((a.N + BN - 1) / BN);

    // codes: offsets from the stage's first token; units past K are out of range, tokens past N past the extent
    const int xt = tid >> 4, xu = tid & 15;
    const bool xk = k0 + 16 * xu < a.K;
    const uint32_t xo = xk ? (uint32_t)(xt * (int)a.ldx + 16 * xu) : OOR;
    const uint32_t so = xk ? (uint32_t)(xt * (int)a.lds + (xu >> 3)) : OOR;
    struct CodeSource {
        __amdgpu_buffer_rsrc_t x, s;
    };
    auto code_source = [&](int s) {
        const int64_t n = (int64_t)s * BN;
        return CodeSource{rsrc(a.X + n * a.ldx + k0, s < S ? (a.N - 1 - n) * a.ldx + a.K - k0 : 0),
                          rsrc(a.xs + n * a.lds + (k0 >> 7), s < S ? (a.N - 1 - n) * a.lds + (a.K + 127) / 128 - (k0 >> 7) : 0)};
    };
    auto load_codes = [&](const CodeSource& src, int h, Codes& c) {
        c.x[h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(src.x, (int)(xo + (xk ? 32u * h * (uint32_t)a.ldx : 0u)), 0, 0));
        c.s[h] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(src.s, (int)(so + (xk ? 32u * h * (uint32_t)a.lds : 0u)), 0, 0);
    };
    // dY: load h of a wave fills tokens 8 wave + 2 h, + 1; lane i the 16 bytes i % 32 of token i / 32, which belong to
    // unit (i % 32) / 2 ^ swz
    uint32_t yo[2];  // by h & 1: swz of tokens 2 h, 2 h + 1 depends on no more, but for bit 3, which is the wave's
#pragma unroll
    for (int v = 0; v < 2; v++) {
        const int n = 8 * wave + 2 * v + (lane >> 5), u = ((lane & 31) >> 1) ^ swz(n);
        yo[v] = (uint32_t)(((lane >> 5) * (int)a.lddy + 16 * u + 8 * (lane & 1)) * 2);
    }
    auto dy_source = [&](int s) {
        const int64_t n = (int64_t)s * BN + 8 * wave;
        const int64_t bytes = ((a.N - 1 - n) * a.lddy + a.M - m0) * 2;
        return make_rsrc(a.dY + (n * a.lddy + m0) * 2, s < S ? (bytes + 3) & ~(int64_t)3 : 0);
    };
    auto load_dy = [&](const i32x4& src, int h, uint32_t buf) {
        dma16(buf + HALF_BYTES + (8 * wave + 2 * h) * 512, yo[h & 1] + (uint32_t)(2 * h * (int)a.lddy * 2), src);
    };
    // half e (8 codes) of unit h, as bf16
    auto write_codes = [&](const Codes& c, int h, int e, uint32_t buf) {
        const int n = xt + 32 * h;
        const float s = scale_value(c.s[h]);
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x[h][2 * e + i], s, false));
            w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x[h][2 * e + i], s, true));
        }
        *(lds_u32x4*)(lds_char*)(size_t)(buf + n * 512 + ((xu ^ swz(n)) << 5) + 16 * e) = w;
    };

    // the lane's place in a step's columns: row 8 q + r / 4, 8 bytes r % 4 of its 32-byte unit; unit c at c ^ swz(row)
    const int row = 8 * q + (r >> 2), rs = swz(row);
    const uint32_t po = (uint32_t)(row * 512 + 8 * (r & 3));
    auto place = [&](int c) { return po + (uint32_t)(((c >> 4) ^ rs) << 5); };
    uint32_t px[FK], py[FM];
#pragma unroll
    for (int i = 0; i < FK; i++) px[i] = place(wk + 16 * i);
#pragma unroll
    for (int j = 0; j < FM; j++) py[j] = HALF_BYTES + place(wm + 16 * j);

    f32x4 acc[FK][FM];
#pragma unroll
    for (int i = 0; i < FK; i++)
#pragma unroll
        for (int j = 0; j < FM; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    Codes c, next;
    {
        const CodeSource c0 = code_source(0), c1 = code_source(1), c2 = code_source(2);
        const i32x4 d0 = dy_source(0), d1 = dy_source(1);
#pragma unroll
        for (int h = 0; h < 2; h++) load_codes(c0, h, c);
#pragma unroll
        for (int h = 0; h < 4; h++) load_dy(d0, h, l0);
#pragma unroll
        for (int h = 0; h < 2; h++) load_codes(c1, h, next);
        __builtin_amdgcn_s_waitcnt(0x0F70);
#pragma unroll
        for (int h = 0; h < 2; h++) write_codes(c, h, 0, l0), write_codes(c, h, 1, l0);
        c = next;
#pragma unroll
        for (int h = 0; h < 4; h++) load_dy(d1, h, l0 + STAGE_BYTES);
#pragma unroll
        for (int h = 0; h < 2; h++) load_codes(c2, h, next);
    }
    __syncthreads();

    bf16x8 x[FK], y0[FM], y1[FM];  // an x fragment is replaced by the next step's after its row of products
#pragma unroll
    for (int i = 0; i < FK; i++) x[i] = frag(l0 + px[i]);
#pragma unroll
    for (int j = 0; j < FM; j++) y0[j] = frag(l0 + py[j]);

    uint32_t cur = l0, oth = l0 + STAGE_BYTES;
#pragma unroll 1
    for (int s = 0; s < S; s++) {
        // step 0, with the fragments of step 1 and the codes of the next stage: side work behind single matrix
        // instructions, so that it runs beside them
#pragma unroll
        for (int i = 0; i < FK; i++)
#pragma unroll
            for (int j = 0; j < FM; j++) {
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y0[j], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                if (j == 0 && i < FM) y1[i] = frag(cur + py[i] + 32 * 512);
                if (j == 2 && i > 0) x[i - 1] = frag(cur + px[i - 1] + 32 * 512);
                if (j == 0 && i >= FM) write_codes(c, (i - FM) >> 1, i & 1, oth);
            }
        x[FK - 1] = frag(cur + px[FK - 1] + 32 * 512);
        __builtin_amdgcn_s_waitcnt(0x0070);  // every load and LDS access of this wave is done
        __builtin_amdgcn_s_barrier();
        // step 1, with the fragments of the next stage's step 0 and the loads of stages s + 2 (dY) and s + 3 (codes)
        const i32x4 dsrc = dy_source(s + 2);
        const CodeSource csrc = code_source(s + 3);
#pragma unroll
        for (int i = 0; i < FK; i++)
#pragma unroll
            for (int j = 0; j < FM; j++) {
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y1[j], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                if (j == 0 && i < FM) y0[i] = frag(oth + py[i]);
                if (j == 2 && i > 0) x[i - 1] = frag(oth + px[i - 1]);
                if (j == 1 && i < 4) load_dy(dsrc, i, cur);
                if (j == 0 && i >= FM && i < FM + 2) {
                    c.x[i - FM] = next.x[i - FM];
                    c.s[i - FM] = next.s[i - FM];
                    load_codes(csrc, i - FM, next);
                }
            }
        x[FK - 1] = frag(oth + px[FK - 1]);
        const uint32_t t = cur;
        cur = oth;
        oth = t;
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // the zero-filling loads past the last stage have landed

    // Four fragments of rows (64 k) at a time: a quad transpose gives each lane quad one row m, 64 consecutive k.
    const int64_t tiles = (a.K + 127) / 128;
    const int xl = r & 3, cq = r >> 2;
    constexpr int W = F32 ? 4 : 2, ES = F32 ? 4 : 2;
#pragma unroll
    for (int j = 0; j < FM; j++)
#pragma unroll
        for (int ig = 0; ig < FK / 4; ig++) {
            uint32_t v[4][W];
#pragma unroll
            for (int f = 0; f < 4; f++) {
                f32x4 y = acc[4 * ig + f][j];
                const int64_t k = k0 + wk + 16 * (4 * ig + f) + 4 * q, m = m0 + wm + 16 * j + r;
                if (a.meta && k < a.K && m < a.M) y = masked(y, a.meta, m, k, tiles);
                if constexpr (F32) {
#pragma unroll
                    for (int e = 0; e < 4; e++) v[f][e] = __float_as_uint(y[e]);
                } else {
                    v[f][0] = pack_bf16x2_rne(y[0], y[1]);
                    v[f][1] = pack_bf16x2_rne(y[2], y[3]);
                }
            }
            slot_transpose4<W>(v, xl);
#pragma unroll
            for (int s = 0; s < 4; s++) {
                const int64_t m = m0 + wm + 16 * j + 4 * cq + s, k = k0 + wk + 64 * ig + 16 * xl + 4 * q;
                if (m < a.M && k < a.K) {
                    char* const p = a.out + (m * a.ldw + k) * ES;
                    if constexpr (F32) __builtin_nontemporal_store(u32x4{v[s][0], v[s][1], v[s][2], v[s][3]}, reinterpret_cast<u32x4*>(p));
                    else __builtin_nontemporal_store(u32x2{v[s][0], v[s][1]}, reinterpret_cast<u32x2*>(p));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
}

}  // namespace

hipError_t launch_grad_weight_tiled(const Fp8GradArgs& g, hipStream_t s) {
    Args a;
    a.dY = static_cast<const char*>(g.dY); a.X = g.X; a.xs = g.xs; a.meta = g.meta; a.out = static_cast<char*>(g.dW);
    a.N = g.N; a.M = g.M; a.K = g.K; a.lddy = g.lddy; a.ldx = g.ldx; a.lds = g.lds; a.ldw = g.ldw;
    a.tilesK = (int)((g.K + BT - 1) / BT);
    a.tilesM = (int)((g.M + BT - 1) / BT);
    const dim3 grid((unsigned)((int64_t)a.tilesK * a.tilesM));
    if (g.out_fp32) hipLaunchKernelGGL((grad_weight_tiled_kernel<true>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((grad_weight_tiled_kernel<false>), grid, dim3(512), 0, s, a);
    return hipGetLastError();
}

}  // namespace sp24
