// Sparse x dense product in 8-bit floating point for many tokens: the launches of the plain product (kernel:
// gemm_fp8_tiled_impl.h).
#include "gemm_fp8_tiled_impl.h"

namespace sp24 {

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
    const bool wide_tiles = rounds >= 4 || narrow > (2 * rounds - 1) * cus;
    if (g.epi.on) return launch_gemm_fp8_tiled_fused(g, wide_tiles, s);
    return wide_tiles ? launch<256>(g, s) : launch<128>(g, s);
}

}  // namespace sp24
