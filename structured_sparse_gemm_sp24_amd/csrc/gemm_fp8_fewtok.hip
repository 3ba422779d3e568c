// Sparse x dense product in 8-bit floating point: the choice of the kernel, and the few-token launches of the plain product
// (kernel: gemm_fp8_fewtok_impl.h).
#include "gemm_fp8_fewtok_impl.h"

namespace sp24 {

hipError_t launch_gemm_fp8(const Fp8GemmArgs& g, hipStream_t s) {
    if (!few_tokens(g)) return launch_gemm_fp8_tiled(g, s);
    return g.epi.on ? launch_gemm_fp8_fewtok_fused(g, s) : launch_fewtok<false>(g, s);
}

}  // namespace sp24
