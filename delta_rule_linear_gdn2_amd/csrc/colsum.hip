// Sums over rows of partial sums: the second step of the weight gradients.
//
// The kernels that produce weight gradients walk many rows each and leave one
// partial row per workgroup (or run of tokens) in the workspace.  Here column c
// is summed over the P partial rows in a fixed order: a workgroup takes 16
// columns (64 bytes a row, one memory segment), its 64 groups of 16 lanes the
// partial rows 64 apart, and the 64 sums meet in LDS.  Narrow tiles, because
// the columns are few: what bounds this is the length of a lane's chain of
// loads.  No atomics, so results repeat bit for bit.
#include "launch.hpp"

namespace gdn2 {
namespace {

constexpr int kCols = 16, kSlices = 64;

__global__ __launch_bounds__(kCols * kSlices) void column_sum_kernel(ColumnSumArgs a)
{
    __shared__ float part[kSlices][kCols + 1];
    const int lane = threadIdx.x % kCols, slice = threadIdx.x / kCols;
    const int64_t c = int64_t(blockIdx.x) * kCols + lane;
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
    if (c < a.width) {
        int64_t r = slice;
        for (; r + 3 * kSlices < a.P; r += 4 * kSlices) {
            s0 += a.partial[r * a.width + c];
            s1 += a.partial[(r + kSlices) * a.width + c];
            s2 += a.partial[(r + 2 * kSlices) * a.width + c];
            s3 += a.partial[(r + 3 * kSlices) * a.width + c];
        }
        for (; r < a.P; r += kSlices) s0 += a.partial[r * a.width + c];
    }
    part[slice][lane] = (s0 + s1) + (s2 + s3);
    __syncthreads();
    if (slice >= 4) return;  // the first wavefront: four lanes a column
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kSlices / 4; ++i) s += part[slice * (kSlices / 4) + i][lane];
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if (slice != 0 || c >= a.width) return;
    int64_t begin = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (c >= begin && c < a.end[i] && a.out[i]) a.out[i][c - begin] = s;
        begin = a.end[i];
    }
}

}  // namespace

hipError_t launch_column_sum(const ColumnSumArgs& a, hipStream_t stream)
{
    const int64_t blocks = (a.width + kCols - 1) / kCols;
    if (blocks == 0) return hipSuccess;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(column_sum_kernel, dim3(unsigned(blocks)), dim3(kCols * kSlices), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn2
