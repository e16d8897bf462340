// sums.hpp -- sums over the parts that workgroups leave in a workspace.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tfla {

// Sums of parts, for a workgroup of 1024 threads: columns block * 64 .. + 63 of part[r * stride + i], i < n, over
// r < parts in a fixed order, 16 slices of the parts side by side.  Returns a column's sum in the threads below 64.
__device__ __forceinline__ float part_sum(const float* __restrict__ part, int64_t parts, int64_t stride, int64_t n,
                                          int64_t block, float (*red)[64])
{
    const int64_t i = block * 64 + (threadIdx.x & 63);
    const int slice = threadIdx.x >> 6;
    float s = 0.0f;
    if (i < n) {
#pragma unroll 4
        for (int64_t r = slice; r < parts; r += 16) s += part[r * stride + i];
    }
    red[slice][threadIdx.x & 63] = s;
    for (int k = 8; k; k >>= 1) {
        __syncthreads();
        if (slice < k) red[slice][threadIdx.x & 63] += red[slice + k][threadIdx.x & 63];
    }
    return red[0][threadIdx.x & 63];
}

}  // namespace tfla
