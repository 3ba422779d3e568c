// Gradient of the fused epilogue: dZ = dY act'(Z), dbias[m] = sum over tokens n of dY act'(Z), one pass over dY and Z.
//
// A thread holds the fp32 sums of eight columns over the rows that it takes, four rows requested at a time; a workgroup adds
// them through LDS, and where the tokens are split into parts a second kernel adds the parts, both in a fixed order.
// HBM bounds it: 8192 x 28672 bf16 286 us, 4.9 TB/s (a large copy reaches 5.1); small ones the launches (64 x 4096 3.5 us).
#include "epilogue.h"

namespace sp24 {
namespace {

constexpr int THREADS = 256;

struct Args {
    const char *dY, *Z;
    char* dZ;
    float* sums;  // dbias, or a row of M partial sums for each part
    int64_t N, M, lddy, ldz, lddz;
    int64_t rows;  // a part's
};

typedef u32x4 u32x4_at2 __attribute__((aligned(2)));

template <int DT, bool ODD>
__device__ __forceinline__ Raw8<DT> load_row8(const char* p, int in) {
    Raw8<DT> r = zero8<DT>();
    if (in == 8) {
        if constexpr (!ODD) return load8_once<DT>(p);
        r.w[0] = *reinterpret_cast<const u32x4_at2*>(p);
        if constexpr (DT == T_FP32) r.w[1] = *reinterpret_cast<const u32x4_at2*>(p + 16);
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (e < in) {
                if constexpr (DT == T_FP32) r.w[e >> 2][e & 3] = reinterpret_cast<const uint32_t*>(p)[e];
                else r.w[0][e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
            }
    }
    return r;
}

template <int DT, bool ODD>
__device__ __forceinline__ void store_row8(char* p, const Raw8<DT>& r, int in) {
    if (in == 8) {
        if constexpr (!ODD) {
            store8<DT>(p, r);
        } else {
            *reinterpret_cast<u32x4_at2*>(p) = r.w[0];
            if constexpr (DT == T_FP32) *reinterpret_cast<u32x4_at2*>(p + 16) = r.w[1];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (e < in) {
                if constexpr (DT == T_FP32) reinterpret_cast<uint32_t*>(p)[e] = r.w[e >> 2][e & 3];
                else reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(r.w[0][e >> 1] >> (16 * (e & 1)));
            }
    }
}

// LANES threads lie along a row, eight columns each, the others on further rows.
template <int DT, int ACT, bool ODD, int LANES>
__global__ __launch_bounds__(THREADS) void epilogue_back_kernel(Args a) {
    constexpr int ES = type_bytes<DT>(), COLS = 8 * LANES, ROWS = THREADS / LANES, UNROLL = 4;
    __shared__ float red[ROWS * COLS];
    const int along = threadIdx.x % LANES, down = threadIdx.x / LANES;
    const int64_t m = (int64_t)blockIdx.x * COLS + 8 * along;
    const int64_t left = a.M - m;
    const int in = left >= 8 ? 8 : left <= 0 ? 0 : (int)left;
    const int64_t n0 = blockIdx.y * a.rows, n1 = n0 + a.rows < a.N ? n0 + a.rows : a.N;
    float sum[8] = {};
    if (in)
        for (int64_t n = n0 + down; n < n1; n += UNROLL * ROWS) {
            Raw8<DT> dy[UNROLL], z[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; u++) {
                const int64_t nu = n + u * ROWS;
                if (nu >= n1) continue;
                dy[u] = load_row8<DT, ODD>(a.dY + (nu * a.lddy + m) * ES, in);
                if constexpr (ACT != ACT_NONE) z[u] = load_row8<DT, ODD>(a.Z + (nu * a.ldz + m) * ES, in);
            }
#pragma unroll
            for (int u = 0; u < UNROLL; u++) {
                const int64_t nu = n + u * ROWS;
                if (nu >= n1) continue;
                float d[8];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    d[e] = ACT == ACT_NONE ? elem<DT>(dy[u], e) : act_back<ACT>(elem<DT>(dy[u], e), elem<DT>(z[u], e));
                    sum[e] += d[e];
                }
                if constexpr (ACT != ACT_NONE) store_row8<DT, ODD>(a.dZ + (nu * a.lddz + m) * ES, pack8<DT>(d), in);
            }
        }
    if (!a.sums) return;
#pragma unroll
    for (int e = 0; e < 8; e++) red[down * COLS + LANES * e + along] = sum[e];
    __syncthreads();
    // column 8 (t % LANES) + t / LANES of the block
    for (int t = threadIdx.x; t < COLS; t += THREADS) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < ROWS; r++) s += red[r * COLS + t];
        const int64_t c = (int64_t)blockIdx.x * COLS + 8 * (t % LANES) + t / LANES;
        if (c < a.M) a.sums[blockIdx.y * a.M + c] = s;
    }
}

// dbias from the parts' sums: 16 columns a workgroup, 16 threads a column, added in a fixed order.
__global__ __launch_bounds__(256) void add_parts_kernel(const float* parts, int count, int64_t M, float* dbias) {
    __shared__ float red[256];
    const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
    const int64_t m = (int64_t)blockIdx.x * 16 + c;
    float s = 0.f;
    if (m < M)
        for (int p = g; p < count; p += 16) s += parts[p * M + m];
    red[threadIdx.x] = s;
    __syncthreads();
    if (g > 0 || m >= M) return;
#pragma unroll
    for (int k = 1; k < 16; k++) s += red[16 * k + c];
    dbias[m] = s;
}

// Threads along a row: pieces of 128 bytes (16-bit types) of many rows, or of a KB. The short ones give more workgroups where rows
// are few or short (short / long, bf16 GELU: 2048 x 4096 15.1 us / 19.9, 6304 x 768 13.0 / 26.8, 513 x 8192 10.4 / 12.0, 400 x 28672 18.8 /
// 20.8), the long ones read long rows faster (8192 x 28672 325 / 288, rows at any element 4096 x 11007 120 / 93, 4096 x 8192 46.9 /
// 44.0; many rows of 5000 to 8191, which the rule leaves to the short ones, too: 4096 x 7168 44 / 40, SiLU 8192 x 5120 63 / 56).
constexpr int LONG = 64, SHORT = 8;

int threads_along(int64_t N, int64_t M) { return M < 8192 || N <= 512 ? SHORT : LONG; }

template <int DT, int ACT>
hipError_t launch(const Args& a, bool odd, int parts, hipStream_t s) {
    const int along = threads_along(a.N, a.M);
    const dim3 grid((unsigned)((a.M + 8 * along - 1) / (8 * along)), (unsigned)parts), block(THREADS);
    if (along == SHORT && odd) hipLaunchKernelGGL((epilogue_back_kernel<DT, ACT, true, SHORT>), grid, block, 0, s, a);
    else if (along == SHORT) hipLaunchKernelGGL((epilogue_back_kernel<DT, ACT, false, SHORT>), grid, block, 0, s, a);
    else if (odd) hipLaunchKernelGGL((epilogue_back_kernel<DT, ACT, true, LONG>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((epilogue_back_kernel<DT, ACT, false, LONG>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_act(const Args& a, int act, bool odd, int parts, hipStream_t s) {
    switch (act) {
    case ACT_GELU: return launch<DT, ACT_GELU>(a, odd, parts, s);
    case ACT_RELU: return launch<DT, ACT_RELU>(a, odd, parts, s);
    case ACT_SILU: return launch<DT, ACT_SILU>(a, odd, parts, s);
    default: return launch<DT, ACT_NONE>(a, odd, parts, s);
    }
}

}  // namespace

// Rows of a part: eight workgroups a compute unit, but two rows a thread at least (512 x 4096 7.9 us against 14.2 with 16, 6304 x 768
// 13.0 / 17.4). Up to eight rows a thread one part, which writes dbias itself: the second launch would take as long (197 x 768 fp32
// 6.0 us).
int64_t part_rows(int64_t N, int64_t M) {
    const int along = threads_along(N, M), down = THREADS / along;
    if (along == SHORT && N <= 8 * down) return N;
    const int64_t cols = (M + 8 * along - 1) / (8 * along), parts = (2048 + cols - 1) / cols, rows = (N + parts - 1) / parts;
    return rows < 2 * down ? 2 * down : (rows + down - 1) / down * down;
}

int epilogue_back_parts(int64_t N, int64_t M) {
    const int64_t rows = part_rows(N, M);
    return (int)((N + rows - 1) / rows);
}

hipError_t launch_epilogue_back(const void* dY, int dtype, int64_t N, int64_t M, int64_t lddy, const void* Z, int64_t ldz, int act,
                                void* dZ, int64_t lddz, float* dbias, void* workspace, hipStream_t s) {
    const int parts = epilogue_back_parts(N, M);
    Args a;
    a.dY = static_cast<const char*>(dY), a.Z = static_cast<const char*>(Z), a.dZ = static_cast<char*>(dZ);
    a.N = N, a.M = M, a.lddy = lddy, a.ldz = ldz, a.lddz = lddz;
    a.rows = part_rows(N, M);
    a.sums = !dbias ? nullptr : parts > 1 ? static_cast<float*>(workspace) : dbias;
    const int64_t es = dtype == T_FP32 ? 4 : 2;
    const bool odd = (lddy * es) % 16 != 0 || (Z && ((ldz * es) % 16 != 0 || (lddz * es) % 16 != 0));
    hipError_t e;
    switch (dtype) {
    case T_BF16: e = launch_act<T_BF16>(a, act, odd, parts, s); break;
    case T_FP16: e = launch_act<T_FP16>(a, act, odd, parts, s); break;
    default: e = launch_act<T_FP32>(a, act, odd, parts, s); break;
    }
    if (e != hipSuccess || !dbias || parts == 1) return e;
    hipLaunchKernelGGL(add_parts_kernel, dim3((unsigned)((M + 15) / 16)), dim3(256), 0, s, static_cast<const float*>(workspace), parts, M, dbias);
    return hipGetLastError();
}

}  // namespace sp24
