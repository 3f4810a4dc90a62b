// Sums the rows of a [rows, cols] float matrix in a fixed order: the second half
// of the backward kernels' reductions over tokens (each CTA of the first half
// leaves one row of partial sums), without atomics, so that a gradient does not
// depend on scheduling.
#include "common.cuh"
#include "kernels.h"
#include "profile.h"

namespace xlstm {
namespace {

// Columns per CTA, threads per column (592 x 2048: 16 columns by 64 threads take 1 us more, 20
// loads of a thread in flight instead of 8 take 3 us more).
constexpr int kCols = 32, kLanes = 32;

// out0 takes the first `split` columns, out1 the others; either may be NULL.
__global__ void __launch_bounds__(kCols * kLanes)
sum_rows_kernel(const float *__restrict__ part, float *__restrict__ out0, float *__restrict__ out1,
                int split, int rows, int cols) {
    __shared__ float red[kLanes][kCols + 1];
    const int col = blockIdx.x * kCols + threadIdx.x;
    float s = 0.f;
    pdl_wait();
    if (col < cols) {
#pragma unroll 8
        for (int r = threadIdx.y; r < rows; r += kLanes) s += part[(size_t)r * cols + col];
    }
    pdl_launch_dependents();
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < cols) {
#pragma unroll
        for (int l = 1; l < kLanes; ++l) s += red[l][threadIdx.x];
        float *out = col < split ? out0 : out1;
        if (out) out[col < split ? col : col - split] = s;
    }
}

}  // namespace

cudaError_t launch_sum_rows(const float *part, float *out0, float *out1, int split, int rows, int cols,
                            cudaStream_t st) {
    KernelTimer timer("sum_rows", st);
    return launch_chained(sum_rows_kernel, dim3((cols + kCols - 1) / kCols), dim3(kCols, kLanes), 0, st, part, out0, out1,
                          split, rows, cols);
}

}  // namespace xlstm
