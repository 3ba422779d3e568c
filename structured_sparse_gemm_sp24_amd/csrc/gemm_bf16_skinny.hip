// Sparse x dense GEMM for few tokens: where it applies, and the launches of the plain product (kernel:
// gemm_bf16_skinny_impl.h).
#include "gemm_bf16_skinny_impl.h"

namespace sp24 {

bool gemm_bf16_skinny_ok(const GemmArgs& g) {
    // 32-bit byte offsets for every element the tiles touch (K padded to 64, plus one tile)
    const int64_t extent = g.tm ? g.N * g.ldx + g.K + 128 : (g.K + 128) * g.ldx;
    return g.N <= 64 && extent * 2 < ((int64_t)1 << 31);
}

hipError_t launch_gemm_bf16_skinny(const GemmArgs& g, hipStream_t s) {
    return g.epi.on ? launch_gemm_bf16_skinny_fused(g, s) : launch_skinny<false>(g, s);
}

}  // namespace sp24
