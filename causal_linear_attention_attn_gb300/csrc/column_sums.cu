// Sums of the columns of a table of partial sums, added in a fixed order: the gradients of vectors and
// matrices that every token shares.  A block takes 32 columns, its eight warps every eighth row each.
#include "internal.h"

namespace la {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps) column_sums_kernel(const __grid_constant__ ColumnSums p) {
  __shared__ float part[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long col = (long)blockIdx.x * 32 + lane;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (col < p.cols) {
    const float *in = p.in + col;
    long r = warp;
    for (; r + 3 * kWarps < p.rows; r += 4 * kWarps)
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += in[(r + u * kWarps) * p.cols];
    for (; r < p.rows; r += kWarps) s[0] += in[r * p.cols];
  }
  part[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (warp || col >= p.cols) return;
  float x = part[0][lane];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) x += part[w][lane];
  long begin = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const auto &q = p.part[i];
    if (col >= begin && col < q.end) {
      const long c = col - begin, D = (q.end - begin) / q.taps;
      if (q.out) q.out[(c % D) * q.taps + c / D] = x;
    }
    begin = q.end;
  }
}

}  // namespace

cudaError_t launch_column_sums(const ColumnSums &p, int kernel_id, cudaStream_t stream) {
  LaunchTimer timer(kernel_id, stream);
  column_sums_kernel<<<(unsigned)((p.cols + 31) / 32), 32 * kWarps, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace la
