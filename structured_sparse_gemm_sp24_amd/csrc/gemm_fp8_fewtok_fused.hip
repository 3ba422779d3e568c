// Sparse x dense product in 8-bit floating point for a few tokens with bias, activation and residual in its epilogue: the
// launches (kernel: gemm_fp8_fewtok_impl.h).
#include "gemm_fp8_fewtok_impl.h"

namespace sp24 {

hipError_t launch_gemm_fp8_fewtok_fused(const Fp8GemmArgs& g, hipStream_t s) { return launch_fewtok<true>(g, s); }

}  // namespace sp24
