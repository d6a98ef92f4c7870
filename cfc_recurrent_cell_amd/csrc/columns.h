// columns.h -- the sums over rows of partial sums that a gradient's workgroups leave
// (layer_norm.hip, short_conv.hip).
#pragma once

#include <hip/hip_runtime.h>

namespace {

// Columns of part [rows, columns] summed in 64 bits, and leave(column, sum) called for each.  32
// columns a workgroup (a cache line of each row), 32 rows at once.
constexpr int kSumCols = 32, kSumRows = 32;
template <class F>
__global__ __launch_bounds__(kSumCols* kSumRows) void column_sums_kernel(const float* __restrict__ part, long long rows,
                                                                         long long columns, F leave) {
    __shared__ double red[kSumRows][kSumCols + 1];
    const int sub = threadIdx.x % kSumCols, slot = threadIdx.x / kSumCols;
    const long long col = (long long)blockIdx.x * kSumCols + sub;
    double x = 0.0;
    if (col < columns)
#pragma unroll 4
        for (long long r = slot; r < rows; r += kSumRows) x += part[r * columns + col];
    red[slot][sub] = x;
    __syncthreads();
    if (slot != 0 || col >= columns) return;
#pragma unroll
    for (int i = 1; i < kSumRows; ++i) x += red[i][sub];
    leave(col, (float)x);
}
template <class F>
void sum_columns(const float* part, long long rows, long long columns, F leave, hipStream_t stream) {
    hipLaunchKernelGGL((column_sums_kernel<F>), dim3((unsigned)((columns + kSumCols - 1) / kSumCols)),
                       dim3(kSumCols * kSumRows), 0, stream, part, rows, columns, leave);
}

}  // namespace
