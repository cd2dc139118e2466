// Parameter gradients from per-work-group partial sums.
#pragma once

#include <hip/hip_runtime.h>

namespace conv3d {
namespace {

constexpr int kSumThreads = 1024, kSumCols = 8, kSumLanes = kSumThreads / kSumCols;

// partial [rows][2][C] -> the column sums of the first C into first, of the
// second into second (either may be null), in fp64 and a fixed order. Latency
// is all there is here: 8 columns (a 32-byte piece of a row) by 128 row lanes
// per work-group, so 1024 rows are 8 loads in flight per thread. (32 columns
// by 8 lanes took 37 us on 1024 x 192 sums, against the 124 us of the pass
// that leaves them.)
__global__ __launch_bounds__(kSumThreads) void column_sums_kernel(const float* partial, int rows,
                                                                  int C, float* first,
                                                                  float* second) {
  __shared__ double part[kSumLanes][kSumCols + 1];
  const int cl = threadIdx.x % kSumCols, lane = threadIdx.x / kSumCols;
  const int col = blockIdx.x * kSumCols + cl;
  double t = 0.0;
  if (col < 2 * C) {
    const float* p = partial + col;
    const long long step = 2LL * C;
    int r = lane;
    for (; r + 7 * kSumLanes < rows; r += 8 * kSumLanes) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = p[(r + k * kSumLanes) * step];
#pragma unroll
      for (int k = 0; k < 8; ++k) t += (double)v[k];
    }
    for (; r < rows; r += kSumLanes) t += (double)p[r * step];
  }
  part[lane][cl] = t;
  __syncthreads();
#pragma unroll
  for (int h = kSumLanes / 2; h > 0; h >>= 1) {
    if (lane < h) part[lane][cl] += part[lane + h][cl];
    __syncthreads();
  }
  if (lane == 0 && col < 2 * C) {
    if (col < C) {
      if (first) first[col] = (float)part[0][cl];
    } else if (second) {
      second[col - C] = (float)part[0][cl];
    }
  }
}

}  // namespace
}  // namespace conv3d
