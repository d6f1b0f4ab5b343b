// kda_colsum.cuh - sums over the rows of a matrix of partial sums, in the rows' order whatever the timing.
#pragma once

#include "kda_internal.cuh"

namespace kda {

constexpr int kSumCols = 32, kSumGroups = 32;

// A block for it: up to 32 groups of threads, as many as there are rows.
inline dim3 sum_block(int rows)
{
    int groups = 1;
    while (groups < rows && groups < kSumGroups) groups *= 2;
    return dim3(kSumCols, (unsigned)groups);
}

// This block's 32 columns from col0 on of part [rows][stride]: group y of the block's n adds the rows y, y + n, ... and the
// groups' sums are added in order. The result is valid in the threads with threadIdx.y == 0.
__device__ __forceinline__ float column_sum(const float *part, int rows, int64_t stride, int col0, int cols, float (&sh)[kSumGroups][kSumCols])
{
    const int c = col0 + threadIdx.x;
    float s = 0.f;
    if (c < cols) {
        const int n = blockDim.y;
        for (int r0 = threadIdx.y; r0 < rows; r0 += 8 * n) {
            float v[8];  // asked for together
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = r0 + i * n < rows ? part[(r0 + i * n) * stride + c] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
    }
    if (blockDim.y == 1) return s;
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0) return 0.f;
    s = 0.f;
#pragma unroll 8
    for (int i = 0; i < (int)blockDim.y; ++i) s += sh[i][threadIdx.x];
    return s;
}

}  // namespace kda
