// Sparse x dense product in 8-bit floating point for many tokens, with a scale for each block of 128.
//
// Workgroup tile 256 (M) x 128 (N), four waves of 128 x 64 = 8 x 4 fragments of v_smfmac_f32_16x16x128_fp8_fp8; two
// workgroups per compute unit (two waves a SIMD), so that one's epilogue and scaling run beside the other's matrix
// instructions. K advances 128 dense columns a stage -- one block of scales, one matrix instruction a fragment --
// through two LDS stage buffers of 36 KB:
//   A (compressed values): one 1 KB tile per 16-row block, already in the operand's lane order;
//   metadata: one 256 B tile per block (lane l's 32-bit index at 4 l);
//   B (codes of X): 128 token rows of 128 bytes; a lane's operand is the two 16-byte units q and q + 4 of its token's
//     row, and unit u of row n is stored at u ^ ((n >> 1) & 7) ^ 4 (n & 1), which keeps the reads free of bank
//     conflicts and each 4 lanes of a load on one 64-byte run.
// A fragment's product of a stage starts from zero, and acc = fma(product, 2^(x scale + w scale), acc): the sums
// over blocks are fp32 sums of exactly scaled terms. The power of two depends on the lane's token and the wave's 128
// rows, so it is formed once for a column of eight fragments.
//
// Loads are buffer loads with LDS destination whose whole byte offset is in the range-checked VGPR operand: rows past
// M and N, 16-byte units past K (inside a row what follows may be NaN codes, which zero weights would not cancel) and
// the loads issued past the workgroup's last tile return zeros.
//
// Persistent: a workgroup walks its tiles (neighbouring tiles on the same XCD at the same time, groups of 8
// tile-rows) with the LDS pipeline continued across tiles.
#include "fp8_device.h"
#include "sp24_launch.h"

namespace sp24 {
namespace {

constexpr int BM = 256, BN = 128, BK = 128, WM = 128, WN = 64, FM = WM / 16, FN = WN / 16;
constexpr int A_BYTES = BM * 64, META_BYTES = BM * 16, B_BYTES = BN * BK;
constexpr int STAGE_BYTES = A_BYTES + META_BYTES + B_BYTES;
constexpr int NBUF = 2;
constexpr int GROUP_M = 8;
constexpr uint32_t OOR = 0x80000000u;  // a byte offset past every record count
static_assert(2 * NBUF * STAGE_BYTES <= 160 * 1024, "two workgroups' stage buffers fit in LDS");

struct Args {
    const uint8_t *values, *meta, *ws, *X, *xs;
    void* Y;
    int64_t M, K, N, ldx, lds, ldy;
    int S;  // stages
    int tilesM, tilesN;
    int y_vec;  // the row pitch allows 8-byte stores
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

// Lane i's 16 bytes land at lds + 16 i; no VGPR is written. Ordered by explicit waits and barriers.
__device__ __forceinline__ void dma16(uint32_t lds, uint32_t voff, const i32x4& rsrc) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(rsrc) : "memory");
}

__device__ __forceinline__ void wait_vmcnt0() { __builtin_amdgcn_s_waitcnt(0x0F70); }
__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

struct Tile {
    int64_t m0, n0;
    bool valid;
};

// Logical tile of workgroup p at its k-th turn (see the int8 kernel's numbering: turn k covers tiles [kG, kG + rem),
// split evenly over the 8 XCDs, workgroup p on XCD p % 8), walked in groups of GROUP_M tile-rows.
__device__ __forceinline__ Tile tile_of(const Args& a, int p, int k) {
    const int G = gridDim.x, T = a.tilesM * a.tilesN;
    const int64_t base = (int64_t)k * G;
    Tile t{0, 0, false};
    if (base >= T) return t;
    const int rem = (T - base) < G ? (int)(T - base) : G;
    const int x = p & 7, i = p >> 3, q8 = rem >> 3, r8 = rem & 7;
    if (i >= q8 + (x < r8 ? 1 : 0)) return t;
    const int L = (int)base + x * q8 + (x < r8 ? x : r8) + i;
    const int gsize = GROUP_M * a.tilesN, g = L / gsize, first = g * GROUP_M;
    const int gm = (a.tilesM - first) < GROUP_M ? (a.tilesM - first) : GROUP_M;
    const int in_g = L - g * gsize;
    t.m0 = (int64_t)(first + in_g % gm) * BM;
    t.n0 = (int64_t)(in_g / gm) * BN;
    t.valid = true;
    return t;
}

// A tile's descriptors: values and metadata of its row blocks, its tokens' scales.
struct Desc {
    i32x4 rA, rM;
    const uint8_t* xs;  // the first token's scales
    int xs_bytes;       // from there to the end of the scales
    const uint8_t* x;  // first token of the wave's rows to load
    int64_t xbytes;    // from there to the end of X, 0 for no tile
    int wrow;          // byte offset of the wave's row of weight scales
};

__device__ __forceinline__ Desc desc_of(const Args& a, const Tile& t, int wave, int wm0) {
    Desc d;
    const int64_t left = (a.M + 15) / 16 - t.m0 / 16, blocks = left < BM / 16 ? left : BM / 16;
    const int64_t tiles = a.S, n1 = t.n0 + (BN / 4) * wave;
    d.rA = make_rsrc(a.values + (t.m0 / 16) * tiles * 1024, t.valid ? blocks * tiles * 1024 : 0);
    d.rM = make_rsrc(a.meta + (t.m0 / 16) * tiles * 256, t.valid ? blocks * tiles * 256 : 0);
    const int64_t sb = (a.N - 1 - t.n0) * a.lds + a.S;
    d.xs = a.xs + t.n0 * a.lds;
    d.xs_bytes = !t.valid ? 0 : (int)(sb > 0x7FFFFFFF ? 0x7FFFFFFF : sb);
    d.x = a.X + n1 * a.ldx;
    d.xbytes = t.valid ? (a.N - 1 - n1) * a.ldx + a.K : 0;
    d.wrow = (int)((t.m0 + wm0) >> 7) * a.S;
    return d;
}

__device__ __forceinline__ int swz(int n) { return ((n >> 1) & 7) ^ ((n & 1) << 2); }

// This wave's share of the loads of stage s: values of row blocks 4 wave .. +3, their metadata, 32 token rows.
struct LoadOffsets {
    uint32_t a, m, b[4];
    int unit[2];  // dense column of the 16-byte unit that load h (parity h & 1) takes
};

__device__ __forceinline__ LoadOffsets load_offsets(const Args& a, int lane) {
    LoadOffsets o;
    o.a = 16 * lane;
    o.m = (uint32_t)((lane >> 4) * a.S * 256 + 16 * (lane & 15));
#pragma unroll
    for (int h = 0; h < 4; h++) {
        const int row = 8 * h + (lane >> 3), u = (lane & 7) ^ swz(row);
        o.b[h] = (uint32_t)(row * (int)a.ldx + 16 * u);
        if (h < 2) o.unit[h] = 16 * u;  // swz depends on h through (4 h) & 7 only
    }
    return o;
}

__device__ __forceinline__ void load_stage(uint32_t lds, const Args& a, const Desc& d, int s, int wave, const LoadOffsets& lo) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int b = 4 * wave + j;
        dma16(lds + b * 1024, lo.a + (uint32_t)(b * a.S + s) * 1024u, d.rA);
    }
    dma16(lds + A_BYTES + 4 * wave * 256, lo.m + (uint32_t)(4 * wave * a.S + s) * 256u, d.rM);
    const int k0 = s * BK, left = (int)a.K - k0;
    const i32x4 rB = make_rsrc(d.x + k0, d.xbytes - k0);
#pragma unroll
    for (int h = 0; h < 4; h++)
        dma16(lds + A_BYTES + META_BYTES + (32 * wave + 8 * h) * 128, lo.unit[h & 1] < left ? lo.b[h] : OOR, rB);
}

typedef __attribute__((address_space(3))) char lds_char;
typedef const __attribute__((address_space(3))) i32x4 lds_i32x4;
typedef const __attribute__((address_space(3))) uint32_t lds_u32;

// An LDS address opaque to the optimizer (keeps the immediates in the reads).
__device__ __forceinline__ const lds_char* stage_addr(uint32_t buf, int off) {
    uint32_t v = buf + (uint32_t)off;
    asm volatile("" : "+v"(v));
    return (const lds_char*)(size_t)v;
}

struct LaneOffsets {
    int a, m, b0, b1;
};

__device__ __forceinline__ i32x8 read_b(uint32_t buf, const LaneOffsets& o, int j) {
    const i32x4 lo = *reinterpret_cast<lds_i32x4*>(stage_addr(buf, o.b0) + j * 2048);
    const i32x4 hi = *reinterpret_cast<lds_i32x4*>(stage_addr(buf, o.b1) + j * 2048);
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// The scales of one stage, as loaded: the lane's token of each fragment column, and the wave's rows.
struct Scales {
    uint32_t x[FN], w;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, bytes, 0x00020000);
}

__device__ __forceinline__ Scales load_scales(const Args& a, const Desc& d, const uint32_t (&off)[FN], int s) {
    Scales r;
    const __amdgpu_buffer_rsrc_t rs = rsrc(d.xs, d.xs_bytes);
    const __amdgpu_buffer_rsrc_t rw = rsrc(a.ws, (int)((a.M + 127) / 128 * a.S));  // below 2^28 (M <= 2^22, K <= 2^20)
#pragma unroll
    for (int j = 0; j < FN; j++) r.x[j] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rs, (int)off[j], s, 0);
    r.w = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rw, d.wrow, s, 0);
    return r;
}

__device__ __forceinline__ void factors(const Scales& s, float (&f)[FN]) {
    const int w = (int)s.w - 127;
#pragma unroll
    for (int j = 0; j < FN; j++) f[j] = __builtin_amdgcn_ldexpf(scale_value(s.x[j]), w);
}

struct AFrags {
    i32x4 a[FM];
    uint32_t idx[FM];
};

__device__ __forceinline__ f32x4 product(const AFrags& fa, int i, const i32x8& b) {
    return __builtin_amdgcn_smfmac_f32_16x16x128_fp8_fp8(fa.a[i], b, f32x4{0.f, 0.f, 0.f, 0.f}, (int)fa.idx[i], 0, 0);
}
__device__ __forceinline__ void add_scaled(f32x4& acc, const f32x4& p, float f) {
#pragma unroll
    for (int e = 0; e < 4; e++) acc[e] = fmaf(p[e], f, acc[e]);
}

__device__ __forceinline__ void column(f32x4 (&acc)[FM][FN], const AFrags& fa, const i32x8& b, int j, float f) {
#pragma unroll
    for (int i = 0; i < FM; i++) add_scaled(acc[i][j], product(fa, i, b), f);
}

// Token-major epilogue from registers: each accumulator is 4 consecutive outputs of token row n. A quad transpose
// across four row fragments gives each lane quad one token row, so a store instruction covers 16 rows x 64 outputs.
template <bool F16, bool FULL>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[FM][FN], const Args& a, int64_t mw, int64_t nw, int lane) {
    const int q = lane >> 4, r = lane & 15, x = r & 3, c = r >> 2;
    uint16_t* const Y = static_cast<uint16_t*>(a.Y);
#pragma unroll
    for (int ig = 0; ig < FM / 4; ig++)
#pragma unroll
        for (int j = 0; j < FN; j++) {
            uint32_t v[4][2];
#pragma unroll
            for (int f = 0; f < 4; f++) {
                const f32x4 y = acc[4 * ig + f][j];
                v[f][0] = pack16<F16>(y[0], y[1]);
                v[f][1] = pack16<F16>(y[2], y[3]);
            }
            slot_transpose4<2>(v, x);
#pragma unroll
            for (int s = 0; s < 4; s++) {
                const int64_t n = nw + 16 * j + 4 * c + s, m = mw + 64 * ig + 16 * x + 4 * q;
                uint16_t* const p = Y + n * a.ldy + m;
                if constexpr (FULL) {
                    __builtin_nontemporal_store(u32x2{v[s][0], v[s][1]}, reinterpret_cast<u32x2*>(p));
                } else if (n < a.N) {
#pragma unroll
                    for (int t = 0; t < 4; t++)
                        if (m + t < a.M) p[t] = (uint16_t)(v[s][t >> 1] >> (16 * (t & 1)));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
}

template <bool F16>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void gemm_fp8_tiled_kernel(Args a) {
    __shared__ __attribute__((aligned(16))) char smem[NBUF * STAGE_BYTES];
    const uint32_t l0 = (uint32_t)(size_t)(lds_char*)smem;
    const int p = blockIdx.x, S = a.S;
    Tile cur = tile_of(a, p, 0);
    if (!cur.valid) return;  // whole workgroup
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wm0 = (wave >> 1) * WM, wn0 = (wave & 1) * WN;
    const LoadOffsets lo = load_offsets(a, lane);
    LaneOffsets o;
    o.a = (wm0 >> 4) * 1024 + lane * 16;
    o.m = A_BYTES + (wm0 >> 4) * 256 + lane * 4;
    o.b0 = A_BYTES + META_BYTES + (wn0 + r) * 128 + 16 * (q ^ swz(r));
    o.b1 = A_BYTES + META_BYTES + (wn0 + r) * 128 + 16 * (q ^ swz(r) ^ 4);
    uint32_t so[FN];
#pragma unroll
    for (int j = 0; j < FN; j++) so[j] = (uint32_t)((wn0 + 16 * j + r) * (int)a.lds);
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    Tile next = tile_of(a, p, 1);
    Desc dc = desc_of(a, cur, wave, wm0), dn = desc_of(a, next, wave, wm0);
    load_stage(l0, a, dc, 0, wave, lo);
    Scales sc = load_scales(a, dc, so, 0);
    wait_vmcnt0();
    __builtin_amdgcn_s_barrier();
    if (S > 1) load_stage(l0 + STAGE_BYTES, a, dc, 1, wave, lo);  // with one stage a workgroup has one tile
    float f[FN];
    factors(sc, f);

    int buf = 0;
    for (int k = 1;; k++) {
        for (int s = 0; s < S; s++, buf ^= 1) {
            const uint32_t cb = l0 + buf * STAGE_BYTES;
            // scales of the next stage (of the next tile after the last), landed by the wait below
            sc = load_scales(a, s + 1 < S ? dc : dn, so, s + 1 < S ? s + 1 : 0);
            AFrags fa;
            const lds_char *pa = stage_addr(cb, o.a), *pm = stage_addr(cb, o.m);
#pragma unroll
            for (int i = 0; i < FM; i++) {
                fa.a[i] = *reinterpret_cast<lds_i32x4*>(pa + i * 1024);
                fa.idx[i] = *reinterpret_cast<lds_u32*>(pm + i * 256);
            }
            i32x8 b0 = read_b(cb, o, 0), b1 = read_b(cb, o, 1);
            __builtin_amdgcn_sched_barrier(0);
            column(acc, fa, b0, 0, f[0]);
            b0 = read_b(cb, o, 2);
            __builtin_amdgcn_sched_barrier(0);
            column(acc, fa, b1, 1, f[1]);
            b1 = read_b(cb, o, 3);
            __builtin_amdgcn_sched_barrier(0);
            wait_lgkmcnt0();  // this wave's reads of the stage are done
            wait_vmcnt0();    // the next stage has landed
            __builtin_amdgcn_s_barrier();
            const bool here = s + NBUF < S;
            load_stage(cb, a, here ? dc : dn, here ? s + NBUF : s + NBUF - S, wave, lo);
            column(acc, fa, b0, 2, f[2]);
            column(acc, fa, b1, 3, f[3]);
            factors(sc, f);
        }
        const int64_t mw = cur.m0 + wm0, nw = cur.n0 + wn0;
        if (mw + WM <= a.M && nw + WN <= a.N && a.y_vec) store_tile<F16, true>(acc, a, mw, nw, lane);
        else store_tile<F16, false>(acc, a, mw, nw, lane);
        if (!next.valid) break;
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        cur = next;
        dc = dn;
        next = tile_of(a, p, k + 1);
        dn = desc_of(a, next, wave, wm0);
    }
    wait_vmcnt0();  // the zero-filling loads past the last tile have landed before the workgroup ends
}

}  // namespace

hipError_t launch_gemm_fp8_tiled(const Fp8GemmArgs& g, hipStream_t s) {
    Args a;
    a.values = g.values; a.meta = g.meta; a.ws = g.ws; a.X = g.X; a.xs = g.xs; a.Y = g.Y;
    a.M = g.M; a.K = g.K; a.N = g.N; a.ldx = g.ldx; a.lds = g.lds; a.ldy = g.ldy;
    a.S = (int)((g.K + BK - 1) / BK);
    a.tilesM = (int)((g.M + BM - 1) / BM);
    a.tilesN = (int)((g.N + BN - 1) / BN);
    a.y_vec = g.ldy % 4 == 0;  // Y is 16-byte aligned
    const int64_t T = (int64_t)a.tilesM * a.tilesN;
    // two workgroups a compute unit walking their tiles; one tile each where a tile has a single stage (the pipeline
    // across tiles needs both buffers within one tile)
    const int cus = device_cus();
    const unsigned grid = (unsigned)(a.S >= NBUF && T > 2 * cus ? 2 * cus : T);
    if (g.out_fp16) hipLaunchKernelGGL((gemm_fp8_tiled_kernel<true>), dim3(grid), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((gemm_fp8_tiled_kernel<false>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace sp24
