// column_sums.hip -- sums of the columns of partial rows, which the kernels
// that make gradients of weights leave behind one a workgroup.
//
// Rows of fp32 are added in fp64, 1024 rows at a time to a workgroup (64
// columns, 16 slices of rows), and the sums of those again until one row is
// left: a fixed order, results reproducible bit for bit.  512 rows of 2560
// columns 4.7 us, 3.4 for a few: the launch and one chain of loads.
#include <algorithm>

#include "kernels.hpp"

namespace selscan {

namespace {

constexpr int kRows = 1024;

// Workgroup (x, y): columns 64 x .. of rows kRows y ..; the first n0 columns of
// the sums go to out0, the others to out1 (NULL: left out), row y of them.
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* part, int64_t n, int64_t n0, int64_t n1, float* out0,
                                                           float* out1, int64_t stride) {
    __shared__ double sm[16][64];
    const int col = threadIdx.x & 63, sl = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + col, all = n0 + n1;
    const int64_t r0 = (int64_t)blockIdx.y * kRows, r1 = min(n, r0 + kRows);
    double v = 0.0;
    if (c < all) {
#pragma unroll 8
        for (int64_t r = r0 + sl; r < r1; r += 16) v += part[r * all + c];
    }
    sm[sl][col] = v;
    __syncthreads();
    if (sl > 0 || c >= all) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) v += sm[i][col];
    float* out = c < n0 ? out0 : out1;
    if (out) out[blockIdx.y * stride + (c < n0 ? c : c - n0)] = (float)v;
}

}  // namespace

// Rows that n partial rows take with the room for their sums behind them.
int64_t column_sums_rows(int64_t n) {
    int64_t rows = n;
    while (n > kRows) rows += n = (n + kRows - 1) / kRows;
    return rows;
}

hipError_t launch_column_sums(float* part, int64_t n, int64_t n0, int64_t n1, float* out0, float* out1, hipStream_t stream) {
    const int64_t all = n0 + n1;
    const unsigned columns = (unsigned)((all + 63) / 64);
    while (n > kRows) {
        const int64_t next = (n + kRows - 1) / kRows;
        float* to = part + n * all;
        hipLaunchKernelGGL(column_sums_kernel, dim3(columns, (unsigned)next), dim3(1024), 0, stream, part, n, n0, n1, to,
                           to + n0, all);
        part = to;
        n = next;
    }
    hipLaunchKernelGGL(column_sums_kernel, dim3(columns), dim3(1024), 0, stream, part, n, n0, n1, out0, out1, 0);
    return hipGetLastError();
}

}  // namespace selscan
