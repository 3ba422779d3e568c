// Sparse x dense product in 8-bit floating point for many tokens, with a scale for each block of 128.
//
// Workgroup tile 256 (M) x 256 (N) with eight waves, or 256 x 128 with four and two workgroups a compute unit; either way two
// waves a SIMD, of 128 x 64 = 8 x 4 fragments of v_smfmac_f32_16x16x128_fp8_fp8, so that one's scaling and epilogue run
// beside the other's matrix instructions. K advances 128 dense columns a stage -- one block of scales, one matrix
// instruction a fragment -- through two LDS stage buffers of 52 or 36 KB:
//   A (compressed values): one 1 KB tile per 16-row block, already in the operand's lane order;
//   metadata: one 256 B tile per block (lane l's 32-bit index at 4 l);
//   B (codes of X): the tile's token rows of 128 bytes; a lane's operand is the two 16-byte units q and q + 4 of its token's
//     row, and unit u of row n is stored at u ^ ((n >> 1) & 7) ^ 4 (n & 1), which keeps the reads free of bank
//     conflicts and each 4 lanes of a load on one 64-byte run.
// The scales ride on the accumulators (Horner's rule). With e_b the exponent of block b's two scales, which depends on
// the lane's token and the wave's 128 rows, an accumulator holds the sum so far in units of 2^e_b: before block b's
// matrix instruction adds its products it is multiplied by 2^(e_(b-1) - e_b), exactly, and the last unit is put back
// in the epilogue. That is four multiplications a fragment and stage; a product from zero and four fused multiply-adds
// into a second accumulator are six instructions and four registers more, and measured 466 us against 392 on 8192^3
// (128-wide tiles both). Accumulators neither overflow nor lose bits this way while a token's units lie within 2^64 of each
// other. Where they do not (the wave keeps the least and the largest), the wave sums that tile again after its last one,
// from memory, adding each block's products with their own scale. Blocks of zeros, whose scale is the least there is, keep
// the unit that they meet and do not count.
//
// Loads are buffer loads with LDS destination whose whole byte offset is in the range-checked VGPR operand: rows past
// M and N, 16-byte units past K (inside a row what follows may be NaN codes, which zero weights would not cancel) and
// the loads issued past the workgroup's last tile return zeros.
//
// The scales themselves are fetched eight stages at a time, a word each, into a buffer of their own.
//
// 28672 x 8192 on 8192 tokens: 1308 to 1339 us (medians of 60 calls in a row; the first ten after a pause take 1410), 2.9
// dense-equivalent PFLOP/s. What bounds it is a SIMD's issue: for each matrix instruction of 16 cycles it issues 6.5 others
// of four, the four multiplications among them, for the most part not beside the other wave's matrix instructions, since the
// stage's barrier keeps the eight waves in step: matrix cores are busy 32 % of the cycles at the 2.0 GHz that the chip holds
// under this load. Those instructions account for 42 cycles a matrix instruction if nothing overlaps; the 50 that the
// counters show leave the rest to the waits at the barrier. HBM is not near: 2.1 GB fetched a call, 1.6 TB/s.
//
// Summing a tile again costs fourteen times the tile: 11008 x 4096 at N = 1500 1100 us where every tile is, against 77.
//
// Persistent: a workgroup walks its tiles (neighbouring tiles on the same XCD at the same time, groups of 8
// tile-rows) with the LDS pipeline continued across tiles.
#include "fp8_device.h"
#include "sp24_launch.h"

namespace sp24 {
namespace {

constexpr int BM = 256, BK = 128, WM = 128, WN = 64, FM = WM / 16, FN = WN / 16;
constexpr int A_BYTES = BM * 64, META_BYTES = BM * 16;
constexpr int NBUF = 2;
constexpr int CHUNK = 8;  // stages whose scales are fetched together

// Tile width: 128 with four waves and two workgroups a compute unit, or 256 with eight waves.
template <int BN_>
struct Cfg {
    static constexpr int BN = BN_, WAVES = BN_ / 32;
    // whether a stage's loads are spread over the matrix instructions after the barrier (28672 x 8192 x 8192:
    // 1379 us against 1414 us in one burst) or issued at once (128 wide, two workgroups a compute unit: 11008 x 4096 at
    // N = 512 35.5 us against 40 us spread), both before the scales' tracking was shortened
    static constexpr bool SPREAD = BN == 256;
    static constexpr int STAGE_BYTES = A_BYTES + META_BYTES + BN * BK;
    static constexpr int CHUNK_BYTES = BN * CHUNK * 4;  // a word for each scale
    static constexpr int LDS_BYTES = NBUF * STAGE_BYTES + 2 * CHUNK_BYTES;
    static_assert((BN == 128 ? 2 : 1) * LDS_BYTES <= 160 * 1024, "the workgroups of a compute unit fit in its LDS");
};
constexpr int GROUP_M = 8;
constexpr uint32_t OOR = 0x80000000u;  // a byte offset past every record count
typedef short i16x2 __attribute__((ext_vector_type(2)));
struct Args {
    const uint8_t *values, *meta, *ws, *X, *xs;
    void* Y;
    int64_t M, K, N, ldx, lds, ldy;
    int S;  // stages
    int tilesM, tilesN;
    int y_vec;  // every row of Y starts on 8 bytes
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

// One byte a lane, zero-extended to the word at lds + 4 i.
__device__ __forceinline__ void dma1(uint32_t lds, uint32_t voff, const i32x4& rsrc) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_ubyte %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(rsrc) : "memory");
}

__device__ __forceinline__ void wait_vmcnt0() { __builtin_amdgcn_s_waitcnt(0x0F70); }
__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

struct Tile {
    int64_t m0, n0;
    bool valid;
};

// Logical tile of workgroup p at its k-th turn (see the int8 kernel's numbering: turn k covers tiles [kG, kG + rem),
// split evenly over the 8 XCDs, workgroup p on XCD p % 8), walked in groups of GROUP_M tile-rows.
template <int BN>
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
    int tokens;         // from the first token to the last of all; those past it take its scales
    const uint8_t* x;  // first token of the wave's rows to load
    int64_t xbytes;    // from there to the end of X, 0 for no tile
    int wrow;          // byte offset of the wave's row of weight scales
};

template <int BN>
__device__ __forceinline__ Desc desc_of(const Args& a, const Tile& t, int wave, int wm0) {
    Desc d;
    const int64_t left = (a.M + 15) / 16 - t.m0 / 16, blocks = left < BM / 16 ? left : BM / 16;
    const int64_t tiles = a.S, n1 = t.n0 + 32 * wave;
    d.rA = make_rsrc(a.values + (t.m0 / 16) * tiles * 1024, t.valid ? blocks * tiles * 1024 : 0);
    d.rM = make_rsrc(a.meta + (t.m0 / 16) * tiles * 256, t.valid ? blocks * tiles * 256 : 0);
    const int64_t sb = (a.N - 1 - t.n0) * a.lds + a.S;
    d.xs = a.xs + t.n0 * a.lds;
    d.tokens = (int)(a.N - 1 - t.n0 < BN ? a.N - 1 - t.n0 : BN);
    d.xs_bytes = !t.valid ? 0 : (int)(sb > 0x7FFFFFFF ? 0x7FFFFFFF : sb);
    d.x = a.X + n1 * a.ldx;
    d.xbytes = t.valid ? (a.N - 1 - n1) * a.ldx + a.K : 0;
    const int64_t m = t.m0 + wm0 < a.M ? t.m0 + wm0 : a.M - 1;
    d.wrow = (int)(m >> 7) * a.S;
    return d;
}

__device__ __forceinline__ int swz(int n) { return ((n >> 1) & 7) ^ ((n & 1) << 2); }

// A wave's share of the loads of a stage: values of 16 / WAVES row blocks, the metadata of four (waves 0 .. 3), 32
// token rows.
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

// The loads of one stage, to be issued one by one (0 .. COUNT - 1) or at once.
template <int BN>
struct StageLoads {
    static constexpr int AL = 16 / Cfg<BN>::WAVES, COUNT = AL + 5;
    static_assert(!Cfg<BN>::SPREAD || COUNT <= FM, "one load a row block");
    uint32_t lds;
    i32x4 rA, rM, rB;
    int s, left, S, wave;

    __device__ __forceinline__ StageLoads(uint32_t lds_, const Args& a, const Desc& d, int s_, int wave_)
        : lds(lds_), rA(d.rA), rM(d.rM), s(s_), left((int)a.K - s_ * BK), S(a.S), wave(wave_) {
        rB = make_rsrc(d.x + s * BK, d.xbytes - s * BK);
    }
    __device__ __forceinline__ void issue(int n, const LoadOffsets& lo) const {
        if (n < AL) {
            const int b = AL * wave + n;
            dma16(lds + b * 1024, lo.a + (uint32_t)(b * S + s) * 1024u, rA);
        } else if (n == AL) {
            if (AL == 4 || wave < 4) dma16(lds + A_BYTES + 4 * wave * 256, lo.m + (uint32_t)(4 * wave * S + s) * 256u, rM);
        } else {
            const int h = n - AL - 1;
            dma16(lds + A_BYTES + META_BYTES + (32 * wave + 8 * h) * 128, lo.unit[h & 1] < left ? lo.b[h] : OOR, rB);
        }
    }
    __device__ __forceinline__ void issue_all(const LoadOffsets& lo) const {
#pragma unroll
        for (int n = 0; n < COUNT; n++) issue(n, lo);
    }
};

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
    int a, m, b0, b1, s;
};

__device__ __forceinline__ i32x8 read_b(uint32_t buf, const LaneOffsets& o, int j) {
    const i32x4 lo = *reinterpret_cast<lds_i32x4*>(stage_addr(buf, o.b0) + j * 2048);
    const i32x4 hi = *reinterpret_cast<lds_i32x4*>(stage_addr(buf, o.b1) + j * 2048);
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// The scales of one stage: the lane's token of each fragment column, and the wave's rows.
struct Scales {
    uint32_t x[FN], w;
};

// Scales of X, CHUNK stages at a time, into one of two LDS areas: a byte load a stage would bring a line of every token
// through L1 each time, which the operands' traffic has emptied by then (8192^3: 460 us). Words
// [token / 8][stage % CHUNK][token % 8]: lane i of a load takes stage i / 8 of token 8 t + i % 8.
__device__ __forceinline__ void load_chunk(uint32_t lds, const Args& a, const Desc& d, int s, int wave, int lane) {
    const i32x4 rS = make_rsrc(d.xs, d.xs_bytes);
#pragma unroll
    for (int h = 0; h < 4; h++) {
        const int t = 4 * wave + h, n = 8 * t + (lane & 7);
        dma1(lds + t * 256, (uint32_t)((n < d.tokens ? n : d.tokens) * (int)a.lds + s + (lane >> 3)), rS);
    }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, bytes, 0x00020000);
}

// The wave's weight scale of stage s of tile d.
__device__ __forceinline__ uint32_t load_w(const Args& a, const Desc& d, int s) {
    const __amdgpu_buffer_rsrc_t rw = rsrc(a.ws, (int)((a.M + 127) / 128 * a.S));  // below 2^28 (M <= 2^22, K <= 2^20)
    return (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rw, d.wrow, s, 0);
}

// The running units of a lane's four tokens, two in a register: exponent of the current one, the least and the largest so
// far (biases included); and the stage's factors 2^(previous - current).
struct Units {
    i16x2 e[FN / 2], lo[FN / 2], hi[FN / 2];
    float f[FN];
    bool apart;  // a block that the running unit cannot hold
};
constexpr int SPAN = 64;

__device__ __forceinline__ void reset(Units& u) {
#pragma unroll
    for (int p = 0; p < FN / 2; p++) u.e[p] = i16x2{0, 0}, u.lo[p] = i16x2{8192, 8192}, u.hi[p] = i16x2{-8192, -8192};
    u.apart = false;
}

// Whether the wave's tile has to be summed block by block.
__device__ __forceinline__ bool far_apart(const Units& u) {
    bool far = u.apart;
#pragma unroll
    for (int j = 0; j < FN; j++) far |= u.hi[j / 2][j % 2] - u.lo[j / 2][j % 2] > SPAN;
    return __builtin_amdgcn_ballot_w64(far) != 0;
}

struct AFrags {
    i32x4 a[FM];
    uint32_t idx[FM];
};

__device__ __forceinline__ void rescale(f32x4& acc, float f) {
#pragma unroll
    for (int e = 0; e < 4; e++) acc[e] *= f;
}

__device__ __forceinline__ void multiply(f32x4& c, const AFrags& fa, int i, const i32x8& b) {
    c = __builtin_amdgcn_smfmac_f32_16x16x128_fp8_fp8(fa.a[i], b, c, (int)fa.idx[i], 0, 0);
}

// Columns 0 and 1 of a stage, one after the other; each fragment is rescaled while the one before is multiplied.
template <int J>
__device__ __forceinline__ void column(f32x4 (&acc)[FM][FN], const AFrags& fa, const i32x8& b, const Units& u) {
#pragma unroll
    for (int i = 0; i < FM; i++) {
        if (i + 1 < FM) rescale(acc[i + 1][J], u.f[J]);
        else rescale(acc[0][J + 1], u.f[J + 1]);
        __builtin_amdgcn_sched_barrier(0);
        multiply(acc[i][J], fa, i, b);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Columns 2 and 3 together, row block by row block; with RELOAD each A fragment is then replaced by the next stage's (at
// pa, pm), so that these reads spread over half a stage.
template <int BN, bool RELOAD>
__device__ __forceinline__ void last_columns(const StageLoads<BN>& loads, const LoadOffsets& lo, f32x4 (&acc)[FM][FN], AFrags& fa, const i32x8& b2, const i32x8& b3,
                                             const Units& u, const lds_char* pa, const lds_char* pm) {
#pragma unroll
    for (int i = 0; i < FM; i++) {
        if constexpr (Cfg<BN>::SPREAD)
            if (i < StageLoads<BN>::COUNT) loads.issue(i, lo);
        rescale(acc[i][3], u.f[3]);
        __builtin_amdgcn_sched_barrier(0);
        multiply(acc[i][2], fa, i, b2);
        __builtin_amdgcn_sched_barrier(0);
        if (i + 1 < FM) rescale(acc[i + 1][2], u.f[2]);
        __builtin_amdgcn_sched_barrier(0);
        multiply(acc[i][3], fa, i, b3);
        if constexpr (RELOAD) {
            fa.a[i] = *reinterpret_cast<lds_i32x4*>(pa + i * 1024);
            fa.idx[i] = *reinterpret_cast<lds_u32*>(pm + i * 256);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Nonzero where one of 16 codes is a number other than zero, or NaN.
__device__ __forceinline__ uint32_t any_code(const i32x4& v) { return (uint32_t)(v[0] | v[1] | v[2] | v[3]) & 0x7F7F7F7Fu; }

__device__ __forceinline__ void read_a(uint32_t buf, const LaneOffsets& o, AFrags& fa) {
    const lds_char *pa = stage_addr(buf, o.a), *pm = stage_addr(buf, o.m);
#pragma unroll
    for (int i = 0; i < FM; i++) {
        fa.a[i] = *reinterpret_cast<lds_i32x4*>(pa + i * 1024);
        fa.idx[i] = *reinterpret_cast<lds_u32*>(pm + i * 256);
    }
}

// What a wave holds of a stage between its parts.
struct Stage {
    AFrags fa;
    i32x8 b0, b1, b2;
    Scales sc;
    Units u;
    int chunk;  // LDS area of the current chunk of scales
};

// The units of a stage whose operands are in `buf` and g. The rare scales are the NaN, which makes the sum NaN, and
// the least one: that of a block of zeros (it keeps the unit) or of numbers below 2^-118 (the sum is made again).
__device__ __forceinline__ void advance(Stage& g, uint32_t buf, const LaneOffsets& o) {
    Units& u = g.u;
    const uint32_t w = g.sc.w;
    i16x2 e[FN / 2], lo[FN / 2], hi[FN / 2];
    uint32_t least = w, most = w, nan = 0;
#pragma unroll
    for (int j = 0; j < FN; j++) least = min(least, g.sc.x[j]), most = max(most, g.sc.x[j]);
#pragma unroll
    for (int p = 0; p < FN / 2; p++) {
        e[p] = __builtin_bit_cast(i16x2, g.sc.x[2 * p] | (g.sc.x[2 * p + 1] << 16)) + __builtin_bit_cast(i16x2, w | (w << 16));
        lo[p] = __builtin_elementwise_min(u.lo[p], e[p]);
        hi[p] = __builtin_elementwise_max(u.hi[p], e[p]);
    }
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(least == 0u || most == 255u) != 0, 0)) {
        uint32_t some = 0;
#pragma unroll
        for (int i = 0; i < FM; i++) some |= any_code(g.fa.a[i]);
        const bool weights = __builtin_amdgcn_ballot_w64(some != 0) != 0;
#pragma unroll
        for (int j = 0; j < FN; j++) {
            const uint32_t x = g.sc.x[j];
            const bool is_nan = max(x, w) == 255u, zero = !is_nan && min(x, w) == 0u;
            const i32x4 first = *reinterpret_cast<lds_i32x4*>(stage_addr(buf, o.b0) + j * 2048);
            const i32x4 last = *reinterpret_cast<lds_i32x4*>(stage_addr(buf, o.b1) + j * 2048);
            u.apart |= zero && weights && any_code(first | last) != 0;
            nan |= (uint32_t)is_nan << j;
            if (is_nan || zero) {
                e[j / 2][j % 2] = u.e[j / 2][j % 2];
                lo[j / 2][j % 2] = u.lo[j / 2][j % 2];
                hi[j / 2][j % 2] = u.hi[j / 2][j % 2];
            }
        }
    }
#pragma unroll
    for (int p = 0; p < FN / 2; p++) {
        const i16x2 d = u.e[p] - e[p];
        u.f[2 * p] = __builtin_amdgcn_ldexpf(1.f, d[0]);
        u.f[2 * p + 1] = __builtin_amdgcn_ldexpf(1.f, d[1]);
        u.e[p] = e[p], u.lo[p] = lo[p], u.hi[p] = hi[p];
    }
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(nan != 0) != 0, 0)) {
#pragma unroll
        for (int j = 0; j < FN; j++) u.f[j] = (nan >> j) & 1u ? __uint_as_float(0x7FC00000u) : u.f[j];
    }
}

__device__ __forceinline__ void read_x_scales(uint32_t area, int off, int s, Scales& sc) {
    const lds_char* p = stage_addr(area + (uint32_t)(s & (CHUNK - 1)) * 32u, off);
#pragma unroll
    for (int j = 0; j < FN; j++) sc.x[j] = *reinterpret_cast<lds_u32*>(p + 512 * j);
}

// Stage s of the current tile from buffer `buf`; its A fragments, first two B columns and scales have been read. Before
// the last two columns the barrier publishes the next stage's buffer and the loads of stage s + 2 (or the next
// tile's) go into this one; a chunk's first stage fetches the next chunk's scales. NEXT: the next stage's operands are
// read in the last two columns; a tile's last stage leaves that to after the epilogue, which needs the registers.
template <int BN, bool NEXT>
__device__ __forceinline__ void stage(const Args& a, const Desc& dc, const Desc& dn, int s, uint32_t l0, int buf,
                                      f32x4 (&acc)[FM][FN], Stage& g, const LaneOffsets& o, int wave, int lane,
                                      const LoadOffsets& lo) {
    constexpr int STAGE_BYTES = Cfg<BN>::STAGE_BYTES, CHUNK_BYTES = Cfg<BN>::CHUNK_BYTES;
    const uint32_t cb = l0 + buf * STAGE_BYTES, nb = l0 + (buf ^ 1) * STAGE_BYTES, chunks = l0 + NBUF * STAGE_BYTES;
    const int S = a.S;
    if ((s & (CHUNK - 1)) == 0) {
        const bool in = s + CHUNK < S;
        load_chunk(chunks + (g.chunk ^ 1) * CHUNK_BYTES, a, in ? dc : dn, in ? s + CHUNK : 0, wave, lane);
    }
    advance(g, cb, o);
    g.sc.w = load_w(a, NEXT ? dc : dn, NEXT ? s + 1 : 0);  // landed by the wait below
    g.b2 = read_b(cb, o, 3);
    rescale(acc[0][0], g.u.f[0]);
    __builtin_amdgcn_sched_barrier(0);
    column<0>(acc, g.fa, g.b0, g.u);
    g.b0 = read_b(cb, o, 2);
    __builtin_amdgcn_sched_barrier(0);
    column<1>(acc, g.fa, g.b1, g.u);
    wait_lgkmcnt0();  // this wave's reads of the stage are done
    wait_vmcnt0();    // the next stage has landed
    __builtin_amdgcn_s_barrier();
    const bool here = s + NBUF < S;
    const StageLoads<BN> loads(cb, a, here ? dc : dn, here ? s + NBUF : s + NBUF - S, wave);
    if constexpr (!Cfg<BN>::SPREAD) loads.issue_all(lo);
    if (!NEXT || ((s + 1) & (CHUNK - 1)) == 0) g.chunk ^= 1;
    read_x_scales(chunks + g.chunk * CHUNK_BYTES, o.s, NEXT ? s + 1 : 0, g.sc);
    if constexpr (NEXT) {
        g.b1 = read_b(nb, o, 0);
        last_columns<BN, true>(loads, lo, acc, g.fa, g.b0, g.b2, g.u, stage_addr(nb, o.a), stage_addr(nb, o.m));
        g.b0 = g.b1;
        g.b1 = read_b(nb, o, 1);
    } else {
        last_columns<BN, false>(loads, lo, acc, g.fa, g.b0, g.b2, g.u, nullptr, nullptr);
    }
}

// How a wave stores its outputs: one by one where it crosses M or N, else eight bytes a lane. Where every row of Y starts on
// eight bytes, non-temporal stores are the faster (28672 x 512 at N = 8192 157 us against 183); elsewhere rows share
// cache lines between waves, and the caches put them together (28671 x 512 228 us against 430; one by one 384; 11007 x 4096
// at N = 1500 80, 90 and 100).
enum { EDGE, EVEN_PITCH, ODD_PITCH };
typedef u32x2 u32x2_any __attribute__((aligned(2)));  // at any element

// Token-major epilogue from registers: each accumulator is 4 consecutive outputs of token row n. A quad transpose
// across four row fragments gives each lane quad one token row, so a store instruction covers 16 rows x 64 outputs.
template <bool F16, int STORE>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[FM][FN], const Units& u, const Args& a, int64_t mw,
                                           int64_t nw, int lane) {
    const int q = lane >> 4, r = lane & 15, x = r & 3, c = r >> 2;
    uint16_t* const Y = static_cast<uint16_t*>(a.Y);
#pragma unroll
    for (int ig = 0; ig < FM / 4; ig++)
#pragma unroll
        for (int j = 0; j < FN; j++) {
            uint32_t v[4][2];
#pragma unroll
            for (int f = 0; f < 4; f++) {
                f32x4 y = acc[4 * ig + f][j];
#pragma unroll
                for (int e = 0; e < 4; e++) y[e] = __builtin_amdgcn_ldexpf(y[e], u.e[j / 2][j % 2] - 254);
                v[f][0] = pack16<F16>(y[0], y[1]);
                v[f][1] = pack16<F16>(y[2], y[3]);
            }
            slot_transpose4<2>(v, x);
#pragma unroll
            for (int s = 0; s < 4; s++) {
                const int64_t n = nw + 16 * j + 4 * c + s, m = mw + 64 * ig + 16 * x + 4 * q;
                uint16_t* const p = Y + n * a.ldy + m;
                if constexpr (STORE == EVEN_PITCH) {
                    __builtin_nontemporal_store(u32x2{v[s][0], v[s][1]}, reinterpret_cast<u32x2*>(p));
                } else if constexpr (STORE == ODD_PITCH) {
                    *reinterpret_cast<u32x2_any*>(p) = u32x2{v[s][0], v[s][1]};
                } else if (n < a.N) {
#pragma unroll
                    for (int t = 0; t < 4; t++)
                        if (m + t < a.M) p[t] = (uint16_t)(v[s][t >> 1] >> (16 * (t & 1)));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
}

// The wave's tile at (mw, nw) from memory: each block's products from zero and added with their own scale, 16 rows at a
// time.
template <bool F16>
__device__ __forceinline__ void sum_apart(const Args& a, int64_t mw, int64_t nw) {
    const int lane = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));  // nothing kept for this
    const int q = lane >> 4, r = lane & 15, S = a.S;
    const int64_t xb = (a.N - 1 - nw) * a.ldx + a.K;
    const __amdgpu_buffer_rsrc_t rX = rsrc(a.X + nw * a.ldx, (int)(xb > 0x7FFFFFFF ? 0x7FFFFFFF : xb));
    const uint8_t* const ws = a.ws + (mw >> 7) * S;
    uint32_t xo[FN], so[FN];
#pragma unroll
    for (int j = 0; j < FN; j++) {
        const int64_t n = 16 * j + r, last = a.N - 1 - nw;
        xo[j] = n <= last ? (uint32_t)(n * a.ldx + 16 * q) : OOR;
        so[j] = (uint32_t)((n <= last ? n : last) * a.lds);
    }
#pragma unroll 1
    for (int i = 0; i < FM && mw + 16 * i < a.M; i++) {
        const uint8_t* const va = a.values + (mw / 16 + i) * S * 1024 + 16 * lane;
        const uint8_t* const ma = a.meta + (mw / 16 + i) * S * 256 + 4 * lane;
        f32x4 acc[FN];
#pragma unroll
        for (int j = 0; j < FN; j++) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int t = 0; t < S; t++) {
            const int left = (int)a.K - t * BK - 16 * q;
            const i32x4 v = *reinterpret_cast<const i32x4*>(va + t * 1024);
            const int idx = *reinterpret_cast<const int*>(ma + t * 256);
            const uint32_t w = ws[t];
#pragma unroll
            for (int j = 0; j < FN; j++) {
                const uint32_t x = (a.xs + nw * a.lds + t)[so[j]], off = xo[j] + (uint32_t)(t * BK);
                const i32x4 lo = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rX, (int)(left > 0 ? off : OOR), 0, 0));
                const i32x4 hi = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rX, (int)(left > 64 ? off + 64u : OOR), 0, 0));
                const i32x8 b = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                const f32x4 p = __builtin_amdgcn_smfmac_f32_16x16x128_fp8_fp8(v, b, f32x4{0.f, 0.f, 0.f, 0.f}, idx, 0, 0);
                const float nan = max(x, w) == 255u ? __uint_as_float(0x7FC00000u) : 0.f;
#pragma unroll
                for (int c = 0; c < 4; c++) acc[j][c] += __builtin_amdgcn_ldexpf(p[c] + nan, (int)(x + w) - 254);
            }
        }
        const int64_t m = mw + 16 * i + 4 * q;
#pragma unroll
        for (int j = 0; j < FN; j++) {
            const int64_t n = nw + 16 * j + r;
            const uint32_t y[2] = {pack16<F16>(acc[j][0], acc[j][1]), pack16<F16>(acc[j][2], acc[j][3])};
            uint16_t* const out = static_cast<uint16_t*>(a.Y) + n * a.ldy + m;
#pragma unroll
            for (int c = 0; c < 4; c++)
                if (n < a.N && m + c < a.M) out[c] = (uint16_t)(y[c >> 1] >> (16 * (c & 1)));
        }
    }
}

template <int BN, bool F16>
__global__ __launch_bounds__(64 * Cfg<BN>::WAVES) __attribute__((amdgpu_waves_per_eu(2, 2))) void gemm_fp8_tiled_kernel(Args a) {
    constexpr int STAGE_BYTES = Cfg<BN>::STAGE_BYTES;
    __shared__ __attribute__((aligned(16))) char smem[Cfg<BN>::LDS_BYTES];
    const uint32_t l0 = (uint32_t)(size_t)(lds_char*)smem;
    const int p = blockIdx.x, S = a.S;
    Tile cur = tile_of<BN>(a, p, 0);
    if (!cur.valid) return;  // whole workgroup
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wm0 = (wave & 1) * WM, wn0 = (wave >> 1) * WN;
    const LoadOffsets lo = load_offsets(a, lane);
    LaneOffsets o;
    o.a = (wm0 >> 4) * 1024 + lane * 16;
    o.m = A_BYTES + (wm0 >> 4) * 256 + lane * 4;
    o.b0 = A_BYTES + META_BYTES + (wn0 + r) * 128 + 16 * (q ^ swz(r));
    o.b1 = A_BYTES + META_BYTES + (wn0 + r) * 128 + 16 * (q ^ swz(r) ^ 4);
    o.s = ((wn0 + r) >> 3) * 256 + (r & 7) * 4;

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    Tile next = tile_of<BN>(a, p, 1);
    Desc dc = desc_of<BN>(a, cur, wave, wm0), dn = desc_of<BN>(a, next, wave, wm0);
    StageLoads<BN>(l0, a, dc, 0, wave).issue_all(lo);
    Stage g;
    g.chunk = 0;
    load_chunk(l0 + NBUF * STAGE_BYTES, a, dc, 0, wave, lane);
    g.sc.w = load_w(a, dc, 0);
    wait_vmcnt0();
    __builtin_amdgcn_s_barrier();
    if (S > 1) StageLoads<BN>(l0 + STAGE_BYTES, a, dc, 1, wave).issue_all(lo);  // with one stage a workgroup has one tile
    reset(g.u);
    read_x_scales(l0 + NBUF * STAGE_BYTES, o.s, 0, g.sc);

    int buf = 0;
    uint64_t apart = 0;  // bit k % 64: the wave's tile k is summed block by block, after the others
    for (int k = 1;; k++) {
        read_a(l0 + buf * STAGE_BYTES, o, g.fa);
        g.b0 = read_b(l0 + buf * STAGE_BYTES, o, 0);
        g.b1 = read_b(l0 + buf * STAGE_BYTES, o, 1);
        for (int s = 0; s < S - 1; s++, buf ^= 1) stage<BN, true>(a, dc, dn, s, l0, buf, acc, g, o, wave, lane, lo);
        stage<BN, false>(a, dc, dn, S - 1, l0, buf, acc, g, o, wave, lane, lo);
        buf ^= 1;
        const int64_t mw = cur.m0 + wm0, nw = cur.n0 + wn0;
        if (__builtin_expect(far_apart(g.u), 0)) apart |= 1ull << ((k - 1) & 63);
        else if (mw + WM > a.M || nw + WN > a.N) store_tile<F16, EDGE>(acc, g.u, a, mw, nw, lane);
        else if (a.y_vec) store_tile<F16, EVEN_PITCH>(acc, g.u, a, mw, nw, lane);
        else store_tile<F16, ODD_PITCH>(acc, g.u, a, mw, nw, lane);
        if (!next.valid) break;
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        reset(g.u);
        cur = next;
        dc = dn;
        next = tile_of<BN>(a, p, k + 1);
        dn = desc_of<BN>(a, next, wave, wm0);
    }
    wait_vmcnt0();  // the zero-filling loads past the last tile have landed before the workgroup ends
    for (int k = 0; apart != 0; k++) {
        const Tile t = tile_of<BN>(a, p, k);
        if (!t.valid) break;
        if ((apart >> (k & 63)) & 1 && t.n0 + wn0 < a.N) sum_apart<F16>(a, t.m0 + wm0, t.n0 + wn0);
    }
}

template <int BN>
hipError_t launch(const Fp8GemmArgs& g, hipStream_t s) {
    Args a;
    a.values = g.values; a.meta = g.meta; a.ws = g.ws; a.X = g.X; a.xs = g.xs; a.Y = g.Y;
    a.M = g.M; a.K = g.K; a.N = g.N; a.ldx = g.ldx; a.lds = g.lds; a.ldy = g.ldy;
    a.S = (int)((g.K + BK - 1) / BK);
    a.tilesM = (int)((g.M + BM - 1) / BM);
    a.tilesN = (int)((g.N + BN - 1) / BN);
    a.y_vec = g.ldy % 4 == 0;  // Y is 16-byte aligned
    const int64_t T = (int64_t)a.tilesM * a.tilesN;
    // as many workgroups as fit walk the tiles; one tile each where a tile has a single stage (the pipeline across
    // tiles needs both buffers within one tile)
    const int fit = (BN == 128 ? 2 : 1) * device_cus();
    const dim3 grid((unsigned)(a.S >= NBUF && T > fit ? fit : T)), block(64 * Cfg<BN>::WAVES);
    if (g.out_fp16) hipLaunchKernelGGL((gemm_fp8_tiled_kernel<BN, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((gemm_fp8_tiled_kernel<BN, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

// Tile width by the rounds of the chip that the tiles take: one 256-wide tile a compute unit, or two 128-wide ones. A round
// of 256-wide tiles is the faster where it is full enough that the 128-wide tiles (half as many columns each) would
// need their last round's second half as well, and from four rounds on, where the two are near each other until the weight no
// longer fits the caches. Measured (us, 128 wide / 256 wide;
// tiles of 256 x 256): 11008 x 4096 at N = 512 (86) 35.6 / 49.5, 700 (129) 56.6 / 58.2, 1024 (172) 57.1 / 52.9, 1500 (258)
// 81.0 / 99.9, 2048 (344) 88.7 / 99.7, 2304 (387) 110.0 / 100.2, 3100 (559) 136.7 / 147.1, 4608 (774) 188.8 / 193.9,
// 6100 (1032) 243.6 / 244.1; 4096 x 4096 at N = 4096 (256) 60.4 / 56.7; 8192 x 8192 at N = 1024 (128) 69.3 / 92.6, 1100 (160)
// 101.3 / 94.0; 6304 x 768 at N = 6304 (625) 43.6 / 52.4; 28672 x 8192 at N = 8192 (3584) 1515 / 1328.
hipError_t launch_gemm_fp8_tiled(const Fp8GemmArgs& g, hipStream_t s) {
    const int64_t cus = device_cus(), m = (g.M + BM - 1) / BM, wide = m * ((g.N + 255) / 256), narrow = m * ((g.N + 127) / 128);
    const int64_t rounds = (wide + cus - 1) / cus;
    return rounds >= 4 || narrow > (2 * rounds - 1) * cus ? launch<256>(g, s) : launch<128>(g, s);
}

}  // namespace sp24
