// Sums over rows of partial sums: the second step of the weight gradients.
//
// The kernels that produce weight gradients walk many rows each and leave one
// partial row per workgroup (or run of tokens) in the workspace.  Here column c
// is summed over the P partial rows in a fixed order: a workgroup of 1024 takes
// COLS columns, its groups of COLS lanes the partial rows in turn, and their sums
// meet in LDS.  No atomics, so results repeat bit for bit.
//
// What bounds it is the length of a lane's chain of loads, as the columns are
// few: 64 columns a workgroup took 9.6 us over 512 rows of 4096, 16 take 5.  Wide
// rows fill the device anyway and want whole 128-byte lines (264 rows of 24576:
// 12 us with 16 columns, 8 with 32).
#include "launch.hpp"

namespace gdn2 {
namespace {

constexpr int kThreads = 1024;

template <int COLS>
__global__ __launch_bounds__(kThreads) void column_sum_kernel(ColumnSumArgs a)
{
    constexpr int kSlices = kThreads / COLS, kParts = 64 / COLS;
    __shared__ float part[kSlices][COLS + 1];
    const int lane = threadIdx.x % COLS, slice = threadIdx.x / COLS;
    const int64_t c = int64_t(blockIdx.x) * COLS + lane;
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
    if (slice >= kParts) return;  // the first wavefront: kParts lanes a column
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kSlices / kParts; ++i) s += part[slice * (kSlices / kParts) + i][lane];
#pragma unroll
    for (int off = COLS; off < 64; off *= 2) s += __shfl_xor(s, off, 64);
    if (slice != 0 || c >= a.width) return;
    int64_t begin = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (c >= begin && c < a.end[i] && a.out[i]) a.out[i][c - begin] = s;
        begin = a.end[i];
    }
}

constexpr int64_t kWide = 8192;  // 256 workgroups of 32 columns

}  // namespace

hipError_t launch_column_sum(const ColumnSumArgs& a, hipStream_t stream)
{
    const int cols = a.width >= kWide ? 32 : 16;
    const int64_t blocks = (a.width + cols - 1) / cols;
    if (blocks == 0) return hipSuccess;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    if (cols == 32)
        hipLaunchKernelGGL(column_sum_kernel<32>, dim3(unsigned(blocks)), dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(column_sum_kernel<16>, dim3(unsigned(blocks)), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn2
