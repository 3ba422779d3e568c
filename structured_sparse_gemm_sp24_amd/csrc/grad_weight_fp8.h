// Shared by the two kernels of the weight's gradient: the 2:4 mask of four consecutive columns.
#pragma once
#include "fp8_device.h"

namespace sp24 {

// v (columns k .. k + 3 of row m, one group) with +0 at the places that the metadata has pruned.
__device__ __forceinline__ f32x4 masked(f32x4 v, const uint8_t* meta, int64_t m, int64_t k, int64_t tiles) {
    const uint32_t byte = meta[tiled_offset<16>(m, k >> 3, tiles)];
    const uint32_t nib = (k & 4) ? byte >> 4 : byte & 15u;
    const uint32_t keep = (1u << (nib & 3u)) | (1u << (nib >> 2));
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] = (keep >> e) & 1u ? v[e] : 0.f;
    return v;
}

}  // namespace sp24
