// Tiled sparse x dense GEMM, token-major, with bias, activation and residual in its epilogue: the launches (kernels:
// gemm_bf16_tiled_impl.h, epilogue.h).
#include "gemm_bf16_tiled_impl.h"

namespace sp24 {

template <int ACT>
static hipError_t launch_act(const GemmArgs& g, bool wide, hipStream_t s) {
    return wide ? launch_bn<true, 256, 1, ACT>(g, s) : launch_bn<true, 128, 2, ACT>(g, s);
}

hipError_t launch_gemm_bf16_fused_tm(const GemmArgs& g, bool wide, hipStream_t s) {
    switch (g.epi.act) {
    case ACT_GELU: return launch_act<ACT_GELU>(g, wide, s);
    case ACT_RELU: return launch_act<ACT_RELU>(g, wide, s);
    case ACT_SILU: return launch_act<ACT_SILU>(g, wide, s);
    default: return launch_act<ACT_NONE>(g, wide, s);
    }
}

}  // namespace sp24
