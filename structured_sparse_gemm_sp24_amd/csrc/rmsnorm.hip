// Root-mean-square norm with the residual's addition and an 8-bit output, its gradients, and the plain conversion
// of an activation to codes and scales.
//
// All three are streams: each element is read once, held in registers between the row's reduction and its use, and
// written once, so HBM bounds them. A row belongs to TPR threads (one wave, or a workgroup), each with C chunks of
// 8 consecutive elements, chunk c of thread t at element 8 (c TPR + t): loads and stores of 16 bytes a lane, and 16
// consecutive lanes hold exactly one block of 128, whose largest magnitude is then four DPP steps.
//
// The norm and its gradients load their rows with the non-temporal hint, which leaves the caches to what is written
// (8192 x 8192 bf16 with the residual, beside a copy's 5.1 TB/s: norm 87 -> 75.6 us, 6.2 TB/s; gradients 107 -> 91.4 us,
// 5.9 TB/s). The quantisation does not gain by it (8191 x 11008 fp16 50.0 -> 51.2 us; 5.4 TB/s).
#include "fp8_device.h"
#include "sp24_launch.h"

namespace sp24 {
namespace {

// Sum over a row's threads: the wave's sum for TPR = 64, else the waves' sums through LDS in wave order. `slot`
// alternates between rows, so one barrier a row is enough: a wave can be at most one row ahead of another.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int slot) {
    v = wave_sum(v);
    if constexpr (TPR == 64) return v;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[slot][wave] = v;
    __syncthreads();
    float s = red[slot][0];
#pragma unroll
    for (int i = 1; i < TPR / 64; i++) s += red[slot][i];
    return s;
}

// The thread's row among its workgroup's, in a scalar register: addresses then are a scalar base and a 32-bit offset.
template <int TPR>
__device__ __forceinline__ int row_of() {
    return TPR == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
}

// One lane's eight values of a block of 128 (16 lanes) as codes, and the block's scale by its first lane. Lanes past
// the row's end hold zeros and store nothing.
__device__ __forceinline__ void store_codes(const float (&y)[8], bool in, uint8_t* codes, uint8_t* scale, int lane) {
    uint32_t big = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const uint32_t a = __float_as_uint(y[e]) & 0x7FFFFFFFu;
        big = a > big ? a : big;
    }
    const uint32_t s = scale_byte(max16(big));
    const float f = code_factor(s);
    if (in) {
        *reinterpret_cast<u32x2*>(codes) = u32x2{codes4(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                                                 codes4(y[4] * f, y[5] * f, y[6] * f, y[7] * f)};
        if ((lane & 15) == 0) *scale = (uint8_t)s;
    }
}

// ---------------------------------------------------------------- quantisation
// One chunk of 8 elements a thread; `per_row` chunks a row, a multiple of 16 so that no block of 128 is cut.
template <int DT>
__global__ __launch_bounds__(256) void quant_kernel(const char* __restrict__ X, int64_t N, int64_t K, int64_t ldx,
                                                    uint32_t per_row, uint8_t* __restrict__ codes, int64_t ldc,
                                                    uint8_t* __restrict__ scales, int64_t lds) {
    const uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t n = (int64_t)(i / per_row);
    const uint32_t c = (uint32_t)(i - (uint64_t)n * per_row);
    const bool in = n < N && 8 * (int64_t)c < K;
    const Raw8<DT> r = in ? load8<DT>(X + (n * ldx + 8 * (int64_t)c) * type_bytes<DT>()) : zero8<DT>();
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; e++) y[e] = elem(r, e);
    store_codes(y, in, codes + n * ldc + 8 * (int64_t)c, scales + n * lds + (c >> 4), threadIdx.x);
}

// ---------------------------------------------------------------- norm
struct NormArgs {
    const char *X, *R, *gamma;
    char* H;
    uint8_t *codes, *scales;
    float* rstd;
    int64_t N, K, ldx, ldr, ldh, ldc, lds;
    float eps;
};

template <int DT, int TPR, int C, bool RES>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void rmsnorm_kernel(NormArgs a) {
    __shared__ float red[2][16];
    constexpr int RPB = TPR == 64 ? 4 : 1, B = type_bytes<DT>();
    const int t = threadIdx.x % TPR;
    const int64_t n = (int64_t)blockIdx.x * RPB + row_of<TPR>();
    if (n >= a.N) return;  // whole waves, and only where no barrier follows (TPR = 64)
    Raw8<DT> x[C], g[C];
    float h[C][8];
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int k = 8 * (c * TPR + t);
        const bool in = k < a.K;
        x[c] = in ? load8_once<DT>(a.X + (n * a.ldx + k) * B) : zero8<DT>();
        if constexpr (RES) {
            const Raw8<DT> r = in ? load8_once<DT>(a.R + (n * a.ldr + k) * B) : zero8<DT>();
            float s[8];
#pragma unroll
            for (int e = 0; e < 8; e++) s[e] = elem(x[c], e) + elem(r, e);
            x[c] = pack8<DT>(s);
        }
        g[c] = in ? load8<DT>(a.gamma + k * B) : zero8<DT>();
    }
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int e = 0; e < 8; e++) {
            h[c][e] = elem(x[c], e);  // the norm and its gradient see the rounded sum that H holds
            sum = fmaf(h[c][e], h[c][e], sum);
        }
    sum = row_sum<TPR>(sum, red, 0);
    const float rstd = 1.0f / sqrtf(sum / (float)a.K + a.eps);
    if (a.rstd && t == 0) a.rstd[n] = rstd;
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int k = 8 * (c * TPR + t);
        const bool in = k < a.K;
        if constexpr (RES)
            if (in) store8<DT>(a.H + (n * a.ldh + k) * B, x[c]);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] = h[c][e] * rstd * elem(g[c], e);
        store_codes(y, in, a.codes + n * a.ldc + k, a.scales + n * a.lds + (k >> 7), t);
    }
}

// ---------------------------------------------------------------- gradients of the norm
struct BackArgs {
    const char *dY, *H, *gamma, *dH;
    const float* rstd;
    char* dX;
    float* part;  // gridDim.x rows of K partial sums of dgamma
    int64_t N, K, lddy, ldh, lddh, lddx;
};

// A workgroup walks rows blockIdx.x * RPB + i, then on by gridDim.x * RPB: with r the row's 1/rms and
// q = r^2 mean(gamma dY h), dX = r (gamma dY - h q) + dH. Each thread keeps the dgamma sums of its own columns in
// registers over all of its rows; the workgroup's sums go to one row of `part`.
template <int DT, int TPR, int C, int WPB, bool RES>
__global__ __launch_bounds__(TPR == 64 ? 64 * WPB : TPR) void rmsnorm_back_kernel(BackArgs a) {
    __shared__ float red[2][16];
    constexpr int RPB = TPR == 64 ? WPB : 1, B = type_bytes<DT>();
    // The widest rows leave a thread too few registers (256) to keep a row's numbers unpacked over the reduction, or
    // dH, or in fp32 gamma: those are read where they are used.
    constexpr bool TIGHT = C == 8, LATE = TIGHT && DT == T_FP32;
    const int t = threadIdx.x % TPR, sub = row_of<TPR>();
    Raw8<DT> g[LATE ? 1 : C];
    float dg[C][8];
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int k = 8 * (c * TPR + t);
        if constexpr (!LATE) g[c] = k < a.K ? load8<DT>(a.gamma + k * B) : zero8<DT>();
#pragma unroll
        for (int e = 0; e < 8; e++) dg[c][e] = 0.f;
    }
    int slot = 0;
    for (int64_t n = (int64_t)blockIdx.x * RPB + sub; n < a.N; n += (int64_t)gridDim.x * RPB, slot ^= 1) {
        const float r = a.rstd[n];
        Raw8<DT> dy[C], h[C], dh[TIGHT ? 1 : C];
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int k = 8 * (c * TPR + t);
            const bool in = k < a.K;
            dy[c] = in ? load8_once<DT>(a.dY + (n * a.lddy + k) * B) : zero8<DT>();
            h[c] = in ? load8_once<DT>(a.H + (n * a.ldh + k) * B) : zero8<DT>();
            if constexpr (RES && !TIGHT) dh[c] = in ? load8_once<DT>(a.dH + (n * a.lddh + k) * B) : zero8<DT>();
        }
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int k = 8 * (c * TPR + t);
            if constexpr (LATE) g[0] = k < a.K ? load8<DT>(a.gamma + k * B) : zero8<DT>();
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float dyh = elem(dy[c], e) * elem(h[c], e);
                sum = fmaf(elem(g[LATE ? 0 : c], e), dyh, sum);
                dg[c][e] = fmaf(dyh, r, dg[c][e]);
            }
            if constexpr (LATE) __builtin_amdgcn_sched_barrier(0);  // the next chunk's gamma not before this one's
        }
        const float q = row_sum<TPR>(sum, red, slot) / (float)a.K * r * r;
        if constexpr (TIGHT)  // unpacked again below
#pragma unroll
            for (int c = 0; c < C; c++) {
                asm volatile("" : "+v"(dy[c].w[0]), "+v"(h[c].w[0]));
                if constexpr (!LATE) asm volatile("" : "+v"(g[c].w[0]));
            }
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int k = 8 * (c * TPR + t), i = LATE ? 0 : c, j = TIGHT ? 0 : c;
            if constexpr (LATE) g[0] = k < a.K ? load8<DT>(a.gamma + k * B) : zero8<DT>();
            if constexpr (TIGHT && RES) {
                dh[0] = k < a.K ? load8_once<DT>(a.dH + (n * a.lddh + k) * B) : zero8<DT>();
            }
            float dx[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                dx[e] = r * fmaf(-elem(h[c], e), q, elem(g[i], e) * elem(dy[c], e));
                if constexpr (RES) dx[e] += elem(dh[j], e);
            }
            if (k < a.K) store8<DT>(a.dX + (n * a.lddx + k) * B, pack8<DT>(dx));
            if constexpr (LATE) __builtin_amdgcn_sched_barrier(0);
        }
    }
    float* const part = a.part + (int64_t)blockIdx.x * a.K;
    if constexpr (TPR == 64) {
        // the waves' sums through LDS, added in wave order
        __shared__ float sums[WPB][512];
        for (int c = 0; c < C; c++) {
            __syncthreads();
#pragma unroll
            for (int cc = 0; cc < C; cc++)
                if (cc == c)
#pragma unroll
                    for (int e = 0; e < 8; e++) sums[sub][e * 64 + t] = dg[cc][e];
            __syncthreads();
            for (int i = threadIdx.x; i < 512; i += 64 * WPB) {
                float s = sums[0][i];
#pragma unroll
                for (int w = 1; w < WPB; w++) s += sums[w][i];
                const int k = 512 * c + 8 * (i & 63) + (i >> 6);
                if (k < a.K) part[k] = s;
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int k = 8 * (c * TPR + t);
            if (k < a.K) {
                *reinterpret_cast<f32x4*>(part + k) = f32x4{dg[c][0], dg[c][1], dg[c][2], dg[c][3]};
                *reinterpret_cast<f32x4*>(part + k + 4) = f32x4{dg[c][4], dg[c][5], dg[c][6], dg[c][7]};
            }
        }
    }
}

// dgamma[k] = sum of `rows` partial sums, 32 columns a workgroup: 32 threads each take every 32nd row of a column,
// then the 32 sums are added in order.
__global__ __launch_bounds__(1024) void dgamma_kernel(const float* __restrict__ part, int rows, int64_t K,
                                                      float* __restrict__ dgamma) {
    __shared__ float s[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t k = (int64_t)blockIdx.x * 32 + x;
    float v = 0.f;
    if (k < K)
        for (int p = y; p < rows; p += 256) {  // eight loads in flight
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = p + 32 * i < rows ? part[(int64_t)(p + 32 * i) * K + k] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; i++) v += w[i];
        }
    s[y][x] = v;
    __syncthreads();
    if (y == 0 && k < K) {
#pragma unroll
        for (int i = 1; i < 32; i++) v += s[i][x];
        dgamma[k] = v;
    }
}

constexpr int WPB = 8;  // waves of a workgroup of the gradient kernel where a row is one wave's

constexpr int64_t kRows = (int64_t)1 << 20;  // rows of one launch: below 2^32 threads at any width

template <int DT, int TPR, int C>
hipError_t launch_norm(NormArgs a, hipStream_t s) {
    constexpr int B = type_bytes<DT>();
    const unsigned rpb = TPR == 64 ? 4 : 1, threads = TPR == 64 ? 256 : TPR;
    for (int64_t left = a.N; left > 0; left -= kRows) {
        a.N = left < kRows ? left : kRows;
        const dim3 grid((unsigned)((a.N + rpb - 1) / rpb));
        if (a.R)
            hipLaunchKernelGGL((rmsnorm_kernel<DT, TPR, C, true>), grid, dim3(threads), 0, s, a);
        else
            hipLaunchKernelGGL((rmsnorm_kernel<DT, TPR, C, false>), grid, dim3(threads), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.X += kRows * a.ldx * B;
        if (a.R) a.R += kRows * a.ldr * B, a.H += kRows * a.ldh * B;
        a.codes += kRows * a.ldc;
        a.scales += kRows * a.lds;
        if (a.rstd) a.rstd += kRows;
    }
    return hipSuccess;
}

// Threads of a row and chunks of a thread by the row's length (us, bf16 with the residual): many rows run alike
// (6304 x 768 with 64 threads x 2 chunks 8.9, with 128 x 1 9.1; 8192 x 4096 with 512 x 1 42.3, with 256 x 2 41.6; 8192 x
// 8192 with 512 x 2 and 256 x 4 76.4; 4096 x 16384 with 1024 x 2 76.8, with 512 x 4 77.4); few are the faster the more
// threads they have (16 x 4096 2.7 against 2.9, 16 x 8192 3.3 against 3.6).
template <int DT>
hipError_t launch_norm_k(const NormArgs& a, hipStream_t s) {
    if (a.K <= 512) return launch_norm<DT, 64, 1>(a, s);
    if (a.K <= 1024) return launch_norm<DT, 64, 2>(a, s);
    if (a.K <= 2048) return launch_norm<DT, 256, 1>(a, s);
    if (a.K <= 4096) return launch_norm<DT, 512, 1>(a, s);
    if (a.K <= 8192) return launch_norm<DT, 512, 2>(a, s);
    if (a.K <= 16384) return launch_norm<DT, 1024, 2>(a, s);
    return launch_norm<DT, 1024, 4>(a, s);
}

template <int DT, int TPR, int C>
hipError_t launch_back(const BackArgs& a, int grid, hipStream_t s) {
    const dim3 threads(TPR == 64 ? 64 * WPB : TPR);
    if (a.dH)
        hipLaunchKernelGGL((rmsnorm_back_kernel<DT, TPR, C, WPB, true>), dim3(grid), threads, 0, s, a);
    else
        hipLaunchKernelGGL((rmsnorm_back_kernel<DT, TPR, C, WPB, false>), dim3(grid), threads, 0, s, a);
    return hipGetLastError();
}

// The same for the gradients: 8192 x 2048 with 256 threads x 1 chunk 30.3 us, with 64 x 4 32.4; 8192 x 8192 with 256 x 4 92.0,
// with 512 x 2 93.7; 4096 x 16384 with 1024 x 2 98, with 512 x 4 99.5; 4096 x 32768 with 512 x 8 220, with 1024 x 4 (whose 128
// registers a thread spill) 632.
template <int DT>
hipError_t launch_back_k(const BackArgs& a, int grid, hipStream_t s) {
    if (a.K <= 512) return launch_back<DT, 64, 1>(a, grid, s);
    if (a.K <= 1024) return launch_back<DT, 64, 2>(a, grid, s);
    if (a.K <= 2048) return launch_back<DT, 256, 1>(a, grid, s);
    if (a.K <= 4096) return launch_back<DT, 256, 2>(a, grid, s);
    if (a.K <= 8192) return launch_back<DT, 256, 4>(a, grid, s);
    if (a.K <= 16384) return launch_back<DT, 1024, 2>(a, grid, s);
    return launch_back<DT, 512, 8>(a, grid, s);
}

template <int DT>
hipError_t launch_quant(const void* X, int64_t N, int64_t K, int64_t ldx, uint8_t* codes, int64_t ldc, uint8_t* scales,
                        int64_t lds, hipStream_t s) {
    const uint32_t per_row = (uint32_t)((K + 127) / 128 * 16);  // at most 2^17
    const int64_t most = ((int64_t)1 << 31) / per_row;          // rows of one launch
    for (int64_t n = 0; n < N; n += most) {
        const int64_t rows = N - n < most ? N - n : most;
        const uint64_t blocks = ((uint64_t)rows * per_row + 255) / 256;
        hipLaunchKernelGGL((quant_kernel<DT>), dim3((unsigned)blocks), dim3(256), 0, s,
                           static_cast<const char*>(X) + n * ldx * type_bytes<DT>(), rows, K, ldx, per_row, codes + n * ldc,
                           ldc, scales + n * lds, lds);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_quant_fp8(const void* X, int dtype, int64_t N, int64_t K, int64_t ldx, uint8_t* codes, int64_t ldc,
                            uint8_t* scales, int64_t lds, hipStream_t s) {
    switch (dtype) {
    case T_BF16: return launch_quant<T_BF16>(X, N, K, ldx, codes, ldc, scales, lds, s);
    case T_FP16: return launch_quant<T_FP16>(X, N, K, ldx, codes, ldc, scales, lds, s);
    default: return launch_quant<T_FP32>(X, N, K, ldx, codes, ldc, scales, lds, s);
    }
}

hipError_t launch_rmsnorm(const void* X, int dtype, int64_t N, int64_t K, int64_t ldx, const void* R, int64_t ldr,
                          const void* gamma, float eps, void* H, int64_t ldh, uint8_t* codes, int64_t ldc,
                          uint8_t* scales, int64_t lds, float* rstd, hipStream_t s) {
    NormArgs a;
    a.X = static_cast<const char*>(X); a.R = static_cast<const char*>(R); a.gamma = static_cast<const char*>(gamma);
    a.H = static_cast<char*>(H); a.codes = codes; a.scales = scales; a.rstd = rstd;
    a.N = N; a.K = K; a.ldx = ldx; a.ldr = ldr; a.ldh = ldh; a.ldc = ldc; a.lds = lds; a.eps = eps;
    switch (dtype) {
    case T_BF16: return launch_norm_k<T_BF16>(a, s);
    case T_FP16: return launch_norm_k<T_FP16>(a, s);
    default: return launch_norm_k<T_FP32>(a, s);
    }
}

// Workgroups (and rows of partial sums) of the gradient kernel: more of them hide more latency, fewer leave fewer partial
// sums (us with 256 / 512 / 1024: 65536 x 768 70.5 / 74.6 / 74.3, 8192 x 4096 57.9 / 50.5 / 55.1, 8192 x 8192 100.8 / 91.1 /
// 97.9, 4096 x 16384 96.5 / 102.5 / 113.8).
int rmsnorm_back_parts(int64_t N, int64_t K) {
    const int64_t rows = K <= 1024 ? (N + WPB - 1) / WPB : N;
    const int64_t most = K <= 1024 || K > 8192 ? 256 : 512;
    return (int)(rows < most ? rows : most);
}

hipError_t launch_rmsnorm_back(const void* dY, int dtype, int64_t N, int64_t K, int64_t lddy, const void* H, int64_t ldh,
                               const float* rstd, const void* gamma, const void* dH, int64_t lddh, void* dX,
                               int64_t lddx, float* dgamma, void* workspace, hipStream_t s) {
    BackArgs a;
    a.dY = static_cast<const char*>(dY); a.H = static_cast<const char*>(H); a.gamma = static_cast<const char*>(gamma);
    a.dH = static_cast<const char*>(dH); a.rstd = rstd; a.dX = static_cast<char*>(dX);
    a.part = static_cast<float*>(workspace);
    a.N = N; a.K = K; a.lddy = lddy; a.ldh = ldh; a.lddh = lddh; a.lddx = lddx;
    const int grid = rmsnorm_back_parts(N, K);
    hipError_t e;
    switch (dtype) {
    case T_BF16: e = launch_back_k<T_BF16>(a, grid, s); break;
    case T_FP16: e = launch_back_k<T_FP16>(a, grid, s); break;
    default: e = launch_back_k<T_FP32>(a, grid, s);
    }
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(dgamma_kernel, dim3((unsigned)((K + 31) / 32)), dim3(1024), 0, s, a.part, grid, K, dgamma);
    return hipGetLastError();
}

}  // namespace sp24
