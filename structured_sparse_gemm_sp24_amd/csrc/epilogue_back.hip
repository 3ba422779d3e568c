// Gradient of the fused epilogue: dZ = dY act'(Z), dbias = its sum over tokens.
#include "epilogue.h"

namespace sp24 {
namespace {

constexpr int WAVES = 4, COLS = 512;  // a workgroup's columns: eight a lane

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

template <int DT, int ACT, bool ODD>
__global__ __launch_bounds__(64 * WAVES) void epilogue_back_kernel(Args a) {
    constexpr int ES = type_bytes<DT>();
    __shared__ float red[(WAVES - 1) * COLS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t m = (int64_t)blockIdx.x * COLS + 8 * lane;
    const int64_t left = a.M - m;
    const int in = left >= 8 ? 8 : left <= 0 ? 0 : (int)left;
    const int64_t n0 = blockIdx.y * a.rows, n1 = n0 + a.rows < a.N ? n0 + a.rows : a.N;
    float sum[8] = {};
    if (in)
        for (int64_t n = n0 + wave; n < n1; n += WAVES) {
            const Raw8<DT> dy = load_row8<DT, ODD>(a.dY + (n * a.lddy + m) * ES, in);
            if constexpr (ACT == ACT_NONE) {
#pragma unroll
                for (int e = 0; e < 8; e++) sum[e] += elem<DT>(dy, e);
            } else {
                const Raw8<DT> z = load_row8<DT, ODD>(a.Z + (n * a.ldz + m) * ES, in);
                float d[8];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    d[e] = act_back<ACT>(elem<DT>(dy, e), elem<DT>(z, e));
                    sum[e] += d[e];
                }
                store_row8<DT, ODD>(a.dZ + (n * a.lddz + m) * ES, pack8<DT>(d), in);
            }
        }
    if (!a.sums) return;
    if (wave > 0) {
#pragma unroll
        for (int e = 0; e < 8; e++) red[(wave - 1) * COLS + 64 * e + lane] = sum[e];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int e = 0; e < 8; e++) {
#pragma unroll
        for (int w = 1; w < WAVES; w++) sum[e] += red[(w - 1) * COLS + 64 * e + lane];
        if (e < in) a.sums[blockIdx.y * a.M + m + e] = sum[e];
    }
}

__global__ __launch_bounds__(256) void add_parts_kernel(const float* parts, int count, int64_t M, float* dbias) {
    const int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (m >= M) return;
    float s = 0.f;
    for (int p = 0; p < count; p++) s += parts[p * M + m];
    dbias[m] = s;
}

template <int DT, int ACT>
hipError_t launch(const Args& a, bool odd, dim3 grid, hipStream_t s) {
    if (odd) hipLaunchKernelGGL((epilogue_back_kernel<DT, ACT, true>), grid, dim3(64 * WAVES), 0, s, a);
    else hipLaunchKernelGGL((epilogue_back_kernel<DT, ACT, false>), grid, dim3(64 * WAVES), 0, s, a);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_act(const Args& a, int act, bool odd, dim3 grid, hipStream_t s) {
    switch (act) {
    case ACT_GELU: return launch<DT, ACT_GELU>(a, odd, grid, s);
    case ACT_RELU: return launch<DT, ACT_RELU>(a, odd, grid, s);
    case ACT_SILU: return launch<DT, ACT_SILU>(a, odd, grid, s);
    default: return launch<DT, ACT_NONE>(a, odd, grid, s);
    }
}

}  // namespace

int epilogue_back_parts(int64_t N, int64_t M) {
    const int64_t cols = (M + COLS - 1) / COLS;
    int64_t parts = (2048 + cols - 1) / cols;
    if (parts > (N + 15) / 16) parts = (N + 15) / 16;
    const int64_t rows = (N + parts - 1) / parts;
    return (int)((N + rows - 1) / rows);
}

hipError_t launch_epilogue_back(const void* dY, int dtype, int64_t N, int64_t M, int64_t lddy, const void* Z, int64_t ldz, int act,
                                void* dZ, int64_t lddz, float* dbias, void* workspace, hipStream_t s) {
    const int parts = epilogue_back_parts(N, M);
    Args a;
    a.dY = static_cast<const char*>(dY), a.Z = static_cast<const char*>(Z), a.dZ = static_cast<char*>(dZ);
    a.N = N, a.M = M, a.lddy = lddy, a.ldz = ldz, a.lddz = lddz;
    a.rows = (N + parts - 1) / parts;
    a.sums = !dbias ? nullptr : parts > 1 ? static_cast<float*>(workspace) : dbias;
    const int64_t es = dtype == T_FP32 ? 4 : 2;
    const bool odd = (lddy * es) % 16 != 0 || (Z && ((ldz * es) % 16 != 0 || (lddz * es) % 16 != 0));
    const dim3 grid((unsigned)((M + COLS - 1) / COLS), (unsigned)parts);
    hipError_t e;
    switch (dtype) {
    case T_BF16: e = launch_act<T_BF16>(a, act, odd, grid, s); break;
    case T_FP16: e = launch_act<T_FP16>(a, act, odd, grid, s); break;
    default: e = launch_act<T_FP32>(a, act, odd, grid, s); break;
    }
    if (e != hipSuccess || !dbias || parts == 1) return e;
    hipLaunchKernelGGL(add_parts_kernel, dim3((unsigned)((M + 255) / 256)), dim3(256), 0, s, static_cast<const float*>(workspace), parts, M, dbias);
    return hipGetLastError();
}

}  // namespace sp24
