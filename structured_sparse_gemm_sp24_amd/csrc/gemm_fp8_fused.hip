// Sparse x dense product in 8-bit floating point for many tokens with bias, activation and residual in its epilogue: the
// launches (kernel: gemm_fp8_tiled_impl.h, epilogue.h).
#include "gemm_fp8_tiled_impl.h"

namespace sp24 {

template <int ACT>
static hipError_t launch_act(const Fp8GemmArgs& g, bool wide, hipStream_t s) {
    return wide ? launch<256, ACT>(g, s) : launch<128, ACT>(g, s);
}

hipError_t launch_gemm_fp8_tiled_fused(const Fp8GemmArgs& g, bool wide, hipStream_t s) {
    switch (g.epi.act) {
    case ACT_GELU: return launch_act<ACT_GELU>(g, wide, s);
    case ACT_RELU: return launch_act<ACT_RELU>(g, wide, s);
    case ACT_SILU: return launch_act<ACT_SILU>(g, wide, s);
    default: return launch_act<ACT_NONE>(g, wide, s);
    }
}

}  // namespace sp24
