// Sparse x dense GEMM for few tokens with bias, activation and residual in its epilogue: the launches (kernel:
// gemm_bf16_skinny_impl.h).
#include "gemm_bf16_skinny_impl.h"

namespace sp24 {

hipError_t launch_gemm_bf16_skinny_fused(const GemmArgs& g, hipStream_t s) { return launch_skinny<true>(g, s); }

}  // namespace sp24
