// Tiled sparse x dense GEMM for large N: the launches of the plain product (kernels: gemm_bf16_tiled_impl.h), and a dense
// reference with the same tiling.
#include "gemm_bf16_tiled_impl.h"

namespace sp24 {
namespace tiled_bf16 {

// ---------------------------------------------------------------- dense reference (measurement only)
// A dense bf16 GEMM on v_mfma_f32_16x16x32_bf16 with the token-major sparse loop's tiling -- 256 x 256 workgroup
// tiles in the same persistent XCD-aware walk, eight waves of 128 x 64, 32 MFMAs per wave per stage, the barrier
// after the first fragment block, the same loads with an SGPR stage offset and the same epilogue -- so that its
// time against the sparse kernel's isolates what 2:4 sparsity changes (a 16 x 16 x 64 block is one smfmac
// instead of two MFMAs). K advances 32 per stage (one MFMA's depth) through four 32 KB stage buffers, about the
// bytes in flight of the sparse loop's three 50 KB ones. The weight is a dense copy in MFMA operand order: tiles
// of 16 rows x 32 columns (1 KB), byte range [16 l, 16 l + 16) = lane l's A operand (row l % 16, columns
// 8 (l / 16) .. +7), stored row block by row block and along K inside a block.
namespace dense_ref {
constexpr int BKD = 32, NB = 4, WAVES = 8, BN = 256;
constexpr int A_TILE = BM * BKD * 2;             // 16 KB
constexpr int STAGE_BYTES = A_TILE + BN * BKD * 2;  // + 256 token rows x 64 B
constexpr int NA = 2, NBL = 2, L = NA + NBL;     // loads per wave per stage (1 KB each)

// The B tile holds 64 B per token row; the 16-byte unit u of row n sits at u ^ ((n >> 2) & 3), so the 16 rows
// of one read group (one unit each) start in 16 distinct 4-bank groups.
struct Tile {
    int64_t m0, n0;
    char* y;
    i32x4 rA, rB;
    bool valid;
};

template <bool OUT_FP32>
__device__ __forceinline__ Tile tile(const Args& a, int L) {
    const TileDesc d = tile_desc<OUT_FP32, BN>(a, L);
    Tile t;
    t.m0 = d.m0;
    t.n0 = d.n0;
    t.y = d.y;
    t.valid = d.valid;
    const int64_t kt = a.K / BKD, blocks_left = (a.M + 15) / 16 - d.m0 / 16;
    const int64_t blocks = blocks_left < BM / 16 ? blocks_left : BM / 16;
    t.rA = make_rsrc(reinterpret_cast<const char*>(a.vals) + (d.m0 / 16) * kt * 1024, d.valid ? blocks * kt * 1024 : 0);
    t.rB = make_rsrc(d.x + d.n0 * a.ldx, d.valid ? ((a.N - 1 - d.n0) * a.ldx + a.K) * 2 : 0);
    return t;
}

template <int k>
__device__ __forceinline__ void load(uint32_t buf, const Tile& t, uint32_t soffA, uint32_t soffB, int wave, uint32_t kt,
                                     uint32_t ldx2, uint32_t la, uint32_t lb) {
    if constexpr (k < NA) {
        const uint32_t b = NA * wave + k;
        dma16s(buf + b * 1024, la + b * kt * 1024u, t.rA, soffA);
    } else {
        const uint32_t r0 = 16 * (NBL * wave + (k - NA));
        dma16s(buf + A_TILE + r0 * 64, lb + r0 * ldx2, t.rB, soffB);
    }
}

template <int k>
__device__ __forceinline__ void loads_at(int slot, uint32_t buf, const Tile& t, uint32_t soffA, uint32_t soffB, int wave,
                                         uint32_t kt, uint32_t ldx2, uint32_t la, uint32_t lb) {
    if constexpr (k < L) {
        if ((k * 3 * FM) / L == slot) load<k>(buf, t, soffA, soffB, wave, kt, ldx2, la, lb);
        loads_at<k + 1>(slot, buf, t, soffA, soffB, wave, kt, ldx2, la, lb);
    }
}

__device__ __forceinline__ bf16x8 read16(uint32_t addr) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(
                                          (const lds_char*)(size_t)stage_addr(addr, 0)));
}

__device__ __forceinline__ void stage(uint32_t l0, uint32_t cur, uint32_t nxt, const Tile& lt, uint32_t ls,
                                      f32x4 (&acc)[FM][4], bf16x8 (&fa)[FM], bf16x8 (&rb)[4], uint32_t oa, uint32_t ob,
                                      int wave, uint32_t kt, uint32_t ldx2, uint32_t la, uint32_t lb) {
    const uint32_t cb = l0 + cur, nb = l0 + nxt;
    rb[2] = read16(cb + ob + 2 * 1024);
    rb[3] = read16(cb + ob + 3 * 1024);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; i++) acc[i][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], rb[0], acc[i][0], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    wait_vmcnt<(NB - 2) * L>();
    __builtin_amdgcn_s_barrier();
    const uint32_t soffA = ls * 1024u, soffB = ls * 64u;
    rb[0] = read16(nb + ob);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; i++) {
        acc[i][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], rb[1], acc[i][1], 0, 0, 0);
        loads_at<0>(i, cb, lt, soffA, soffB, wave, kt, ldx2, la, lb);
        __builtin_amdgcn_sched_barrier(0);
    }
    rb[1] = read16(nb + ob + 1024);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; i++) {
        acc[i][2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], rb[2], acc[i][2], 0, 0, 0);
        loads_at<0>(FM + i, cb, lt, soffA, soffB, wave, kt, ldx2, la, lb);
        __builtin_amdgcn_sched_barrier(0);
    }
    const lds_char* pa = (const lds_char*)(size_t)stage_addr(nb, oa);
#pragma unroll
    for (int i = 0; i < FM; i++) {
        acc[i][3] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], rb[3], acc[i][3], 0, 0, 0);
        fa[i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(pa + i * 1024));
        loads_at<0>(2 * FM + i, cb, lt, soffA, soffB, wave, kt, ldx2, la, lb);
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <bool OUT_FP32>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(2, 2))) void gemm_dense_kernel(Args a) {
    constexpr int SB = STAGE_BYTES;
    __shared__ __attribute__((aligned(16))) char smem[NB * SB];
    const uint32_t l0 = (uint32_t)(size_t)(__attribute__((address_space(3))) char*)smem;
    const int p = blockIdx.x;
    int Lt = tile_of(a, p, 0);
    if (Lt < 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm0 = (wave / (WAVES / 2)) * WM, wn0 = (wave % (WAVES / 2)) * 64;
    const int r = lane & 15, q = lane >> 4;
    // LDS read offsets: A fragment i of the wave at (wm0 / 16 + i) KB + 16 lane; B fragment j at token row
    // wn0 + 16 j + r, unit q (swizzled)
    const uint32_t oa = (uint32_t)((wm0 >> 4) * 1024 + lane * 16);
    const uint32_t ob = (uint32_t)(A_TILE + (wn0 + r) * 64 + 16 * (q ^ ((r >> 2) & 3)));
    // load offsets (the range-checked lane part): A 16 lane; B row lane / 4 of a 16-row group, unit lane % 4 of
    // that row's swizzled order
    const uint32_t la = (uint32_t)(16 * lane);
    const uint32_t lb = (uint32_t)((lane >> 2) * a.ldx * 2 + 16 * ((lane & 3) ^ ((lane >> 4) & 3)));
    const int S = (int)(a.K / BKD);
    const uint32_t kt = (uint32_t)S, ldx2 = (uint32_t)(a.ldx * 2);

    f32x4 acc[FM][4];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    Tile cur_t = tile<OUT_FP32>(a, Lt);
    Tile nxt_t = tile<OUT_FP32>(a, tile_of(a, p, 1));
#pragma unroll
    for (int i = 0; i < NB; i++) {
        const bool here = i < S;
        const uint32_t ls = here ? i : i - S;
        if (i == NB - 1) {
            wait_vmcnt<(NB - 2) * L>();
            __builtin_amdgcn_s_barrier();
        }
#pragma unroll
        for (int k = 0; k < L; k++) {
            const Tile& t = here ? cur_t : nxt_t;
            if (k == 0) load<0>(i * SB, t, ls * 1024u, ls * 64u, wave, kt, ldx2, la, lb);
            if (k == 1) load<1>(i * SB, t, ls * 1024u, ls * 64u, wave, kt, ldx2, la, lb);
            if (k == 2) load<2>(i * SB, t, ls * 1024u, ls * 64u, wave, kt, ldx2, la, lb);
            if (k == 3) load<3>(i * SB, t, ls * 1024u, ls * 64u, wave, kt, ldx2, la, lb);
        }
    }
    bf16x8 fa[FM], rb[4];
#pragma unroll
    for (int i = 0; i < FM; i++) fa[i] = read16(l0 + oa + i * 1024);
    rb[0] = read16(l0 + ob);
    rb[1] = read16(l0 + ob + 1024);
    uint32_t cur = 0;
    for (int k = 1;; k++) {
        int s = 0;
        for (; s < S - NB; s++) {
            const uint32_t nxt = cur == (NB - 1) * SB ? 0u : cur + SB;
            stage(l0, cur, nxt, cur_t, (uint32_t)(s + NB), acc, fa, rb, oa, ob, wave, kt, ldx2, la, lb);
            cur = nxt;
        }
        for (; s < S; s++) {
            const uint32_t nxt = cur == (NB - 1) * SB ? 0u : cur + SB;
            stage(l0, cur, nxt, nxt_t, (uint32_t)(s + NB - S), acc, fa, rb, oa, ob, wave, kt, ldx2, la, lb);
            cur = nxt;
        }
        {
            const int64_t mw = cur_t.m0 + wm0, nw = cur_t.n0 + wn0;
            if ((mw + WM <= a.M) && (nw + 64 <= a.N) && a.y_vec)
                store_tile_tm<OUT_FP32, true>(acc, a, cur_t.y, mw, nw, lane);
            else
                store_tile_tm<OUT_FP32, false>(acc, a, cur_t.y, mw, nw, lane);
        }
        if (!nxt_t.valid) break;
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        cur_t = nxt_t;
        nxt_t = tile<OUT_FP32>(a, tile_of(a, p, k + 1));
    }
    wait_vmcnt<0>();
}

// Dense M x K bf16 (row pitch ldw) -> the tiled operand order above; rows past M padded with zeros. One thread
// per 16-byte chunk of the output.
__global__ __launch_bounds__(256) void dense_tile_kernel(const uint16_t* __restrict__ W, int64_t M, int64_t K, int64_t ldw,
                                                         u32x4* __restrict__ out, int64_t chunks) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= chunks) return;
    const int64_t kt = K / BKD;
    const int l = (int)(c & 63);
    const int64_t t = (c >> 6) % kt, b = (c >> 6) / kt;
    const int64_t m = 16 * b + (l & 15), k = BKD * t + 8 * (l >> 4);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (m < M) v = *reinterpret_cast<const u32x4*>(W + m * ldw + k);
    out[c] = v;
}
}  // namespace dense_ref

}  // namespace tiled_bf16

bool gemm_bf16_tiled_ok(const GemmArgs& g) {
    // 32-bit load offsets stay below bit 31, which marks the loads past the last tile: 64 rows of X
    // (64 * ldx * 2), token-major 256 rows (256 * ldx * 2), and 16 row blocks of compressed tiles
    // (16 * K / 64 * 1 KB); 16-byte aligned rows of X in every batch entry
    const bool x_ok = g.ldx % 8 == 0 && (reinterpret_cast<uintptr_t>(g.X) & 15) == 0 && (g.batch == 1 || g.sx % 8 == 0);
    const bool tm_ok = !g.tm || (g.K % 64 == 0 && g.ldx < ((int64_t)1 << 22));
    const int64_t tiles = ((g.M + 255) / 256) * ((g.N + 127) / 128) * g.batch;
    return x_ok && tm_ok && g.N > 64 && g.ldx < ((int64_t)1 << 24) && g.K < ((int64_t)1 << 22) && tiles < (1 << 30);
}

// Number of compute units of the current device (cached per device).
int device_cus() {
    static int cached[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (cached[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
        cached[dev] = n;
    }
    return cached[dev];
}

// Tile width for a launch of the tiled int8 GEMM (either layout). A 128-wide tile costs about C128 of
// a 256-wide one (measured on MI355X), so it wins when the 256-wide tiles leave a last partial turn that
// the 128-wide ones fill better: e.g. 3072 x 8192 has 384 tiles of 256 x 256 on 256 compute units (two
// turns), and 768 of 256 x 128 (three turns of the cheaper tile).
int tiled_tile_width(const GemmArgs& g) {
    constexpr double C128 = 0.6;
    const int64_t cus = device_cus();
    const int64_t tm = (g.M + 255) / 256;
    const int64_t t256 = tm * ((g.N + 255) / 256) * g.batch, t128 = tm * ((g.N + 127) / 128) * g.batch;
    const double c256 = (double)((t256 + cus - 1) / cus), c128 = C128 * (double)((t128 + cus - 1) / cus);
    return c128 < c256 ? 128 : 256;
}

// Configuration of a bf16 launch, measured on MI355X (bit-identical results: the K order inside a tile does
// not depend on the tile shape):
//  - from 32 stages (K >= 2048) 256 x 256 tiles, unless they would leave more than three quarters of the CUs
//    idle: a workgroup of 256 x 128 alone on its CU runs its single wave per SIMD latency-bound, and two of
//    them share the loads of a 256 x 256 tile less well (token-major, against the rule below: 28672 x 8192 x
//    512 144.8 -> 128.0 us, 11008 x 4096 x 1024 58.0 -> 53.1, 3072 x 4096 x 6304 106.5 -> 100.3, 16384 x 8192
//    x 512 113.7 -> 108.6, 768 x 3072 x 8192 32.9 either way; feature-major 28672 x 8192 x 512 146.2 -> 143.7);
//  - below that, 256 x 128 tiles with two workgroups per CU fill the CUs better when there are fewer 256 x 256 tiles
//    than CUs, and fill a partial last turn better: their last turn's tiles run one per CU, at about 0.6
//    of a paired turn, while a full turn of 256 x 256 tiles costs about 0.92 of one (3072 x 768 x 6304
//    token-major: 26.4 us against 30.8 with 256 x 256);
//  - 256 x 256 tiles otherwise (a full first turn, or more than two turns): token-major with eight waves per
//    workgroup, two per SIMD, so the big tile's re-use stays and a second wave covers each one's barrier
//    and load waits (11008 x 4096 x 4096: 235.4 -> 212.2 us against four waves; 28672 x 8192 x 8192:
//    2115 -> 1986 us; against 256 x 128 two per CU: 4096^3 90.8 -> 83.7 us, 4096 x 4096 x 8192 160 -> 152,
//    4096 x 2048 x 8192 101 -> 91); feature-major with four waves (its eight-wave build spills registers;
//    4096^3 82.4 -> 77.7 us).
hipError_t launch_gemm_bf16_tiled(const GemmArgs& g, hipStream_t s) {
    const int64_t tm = ((g.M + 255) / 256) * g.batch, cus = device_cus();
    const int64_t t256 = tm * ((g.N + 255) / 256), t128 = tm * ((g.N + 127) / 128);
    // turns of each tiling in units of a paired 256 x 128 turn
    const double c256 = 0.92 * (double)((t256 + cus - 1) / cus);
    const int64_t rem = t128 % (2 * cus);
    const double c128 = (double)(t128 / (2 * cus)) + (rem == 0 ? 0.0 : rem <= cus ? 0.6 : 1.0);
    const int64_t stages = (g.K + tiled_bf16::BK - 1) / tiled_bf16::BK;
    const bool wide = (stages >= 32 && 4 * t256 >= cus) || !(t256 < cus || (t256 <= 2 * cus && c128 <= c256));
    if (g.epi.on && g.tm) return launch_gemm_bf16_fused_tm(g, wide, s);
    // Feature-major with a fused epilogue (us, 128 wide / 256 wide, bias and GELU): the four waves of a 256-wide tile are alone on their
    // SIMDs in the epilogue, while of two 128-wide workgroups one can multiply meanwhile: 512 x 128 over 32 x 784 26 / 34, 2048 x
    // 2048 over 4 x 3136 (416 wide tiles) 93 / 107; a single turn of wide tiles over a long K 4096 x 4096 over 4096 90 / 85,
    // 28672 x 8192 over 512 157 / 150.
    if (g.epi.on) return launch_gemm_bf16_fused_fm(g, wide && stages >= 32 && t256 <= cus, s);
    if (wide) return g.tm ? launch_bn<true, 256, 1>(g, s) : launch_bn<false, 256, 1>(g, s);
    return g.tm ? launch_bn<true, 128, 2>(g, s) : launch_bn<false, 128, 2>(g, s);
}

}  // namespace sp24

namespace sp24 {

// Host side of the dense reference (measurement only; arguments validated by the C ABI).
hipError_t launch_dense_tile(const void* W, int64_t M, int64_t K, int64_t ldw, void* Wt, hipStream_t s) {
    const int64_t chunks = (M + 15) / 16 * (K / tiled_bf16::dense_ref::BKD) * 64;
    hipLaunchKernelGGL(tiled_bf16::dense_ref::dense_tile_kernel, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, s,
                       static_cast<const uint16_t*>(W), M, K, ldw, static_cast<u32x4*>(Wt), chunks);
    return hipGetLastError();
}

hipError_t launch_gemm_dense_ref(const GemmArgs& g, hipStream_t s) {
    namespace D = tiled_bf16::dense_ref;
    tiled_bf16::Args a;
    a.vals = static_cast<const uint16_t*>(g.values); a.meta = nullptr;
    a.X = static_cast<const uint16_t*>(g.X); a.Y = g.Y;
    a.M = g.M; a.K = g.K; a.N = g.N; a.ldx = g.ldx; a.ldy = g.ldy;
    a.sxb = 0; a.syb = 0;
    a.tilesM = (int)((g.M + tiled_bf16::BM - 1) / tiled_bf16::BM);
    a.tilesN = (int)((g.N + D::BN - 1) / D::BN);
    a.batch = 1;
    const int64_t es = g.out_fp32 ? 4 : 2;
    a.y_vec = ((reinterpret_cast<uintptr_t>(g.Y) & 15) == 0) && ((g.ldy * es) % 16 == 0) && g.ldy * es * 16 < ((int64_t)1 << 31);
    const int T = a.tilesM * a.tilesN;
    const int S = (int)(g.K / D::BKD);
    const int slots = device_cus();
    const unsigned grid = (unsigned)(S >= D::NB && T > slots ? slots : T);
    if (g.out_fp32)
        hipLaunchKernelGGL((D::gemm_dense_kernel<true>), dim3(grid), dim3(64 * D::WAVES), 0, s, a);
    else
        hipLaunchKernelGGL((D::gemm_dense_kernel<false>), dim3(grid), dim3(64 * D::WAVES), 0, s, a);
    return hipGetLastError();
}

}  // namespace sp24
