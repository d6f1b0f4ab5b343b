// kda_colsum.cuh - sums over the rows of a matrix of partial sums, in the rows' order whatever the timing.
#pragma once

#include "kda_internal.cuh"

namespace kda {

constexpr int kSumCols = 32, kSumGroups = 32;

// This block's 32 columns from col0 on of part [rows][stride]: group y of the block adds the rows y, y + 32, ... and the
// groups' sums are added in order. The result is valid in the threads with threadIdx.y == 0.
__device__ __forceinline__ float column_sum(const float *part, int rows, int64_t stride, int col0, int cols, float (&sh)[kSumGroups][kSumCols])
{
    const int c = col0 + threadIdx.x;
    float s = 0.f;
    if (c < cols)
#pragma unroll 4
        for (int r = threadIdx.y; r < rows; r += kSumGroups) s += part[r * stride + c];
    __syncthreads();
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumGroups; ++i) s += sh[i][threadIdx.x];
    return s;
}

}  // namespace kda
