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

// A value that the group's are counted from: of its first and one in its middle
// the one of lesser magnitude (an outlier among them is not taken), or 0 where
// their signs differ. It lies between the group's least and greatest value, so
// what is left is of the size of their spread. x: the group's first value in
// its unit, of P pixels and cpg channels. (Four values: [1,5,16,16,1024] bf16
// forward 7.7 instead of 7.5 us.)
template <class T>
struct Samples {
  typename T::store v[2];
  __device__ __forceinline__ void load(const typename T::store* x, long long P, long long pitch,
                                       int cpg) {
    v[0] = x[0];
    v[1] = x[P / 2 * pitch + cpg / 2];
  }
  __device__ __forceinline__ float reference() const {
    const float k = T::get(v[0]), s = T::get(v[1]);
    return (k < 0.0f) != (s < 0.0f) ? 0.0f : fabsf(s) < fabsf(k) ? s : k;
  }
};

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
