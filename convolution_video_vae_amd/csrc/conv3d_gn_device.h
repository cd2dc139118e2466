// Device helpers of the training GroupNorm kernels.
#pragma once

#include <hip/hip_runtime.h>

namespace conv3d {
namespace {

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// rstd (gamma da - c1 - h c2), each product rounded on its own: the three
// terms cancel where a group holds few values, and to exactly zero where it
// holds one.
__device__ __forceinline__ float gn_dx(float rstd, float gamma, float da, float c1, float h,
                                       float c2) {
#pragma clang fp contract(off)
  const float t = gamma * da;
  const float s = h * c2;
  return rstd * (t - c1 - s);
}

}  // namespace
}  // namespace conv3d
