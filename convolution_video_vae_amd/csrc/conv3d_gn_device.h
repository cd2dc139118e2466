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

// A value that the group's are counted from, out of four of them: the one of
// least magnitude, or 0 where their signs differ. Where all values lie far from
// zero it is one of them, and what is left is of the size of their spread; an
// outlier is not taken. x: the group's first value in its unit, of P pixels and
// cpg channels.
template <class T>
struct Samples {
  typename T::store v[4];
  __device__ __forceinline__ void load(const typename T::store* x, long long P, long long pitch,
                                       int cpg) {
    v[0] = x[0];
    v[1] = x[P / 3 * pitch + cpg / 2];
    v[2] = x[(P - 1 - P / 3) * pitch + cpg / 3];
    v[3] = x[(P - 1) * pitch + cpg - 1];
  }
  __device__ __forceinline__ float reference() const {
    float k = T::get(v[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      const float s = T::get(v[i]);
      k = (k < 0.0f) != (s < 0.0f) ? 0.0f : fabsf(s) < fabsf(k) ? s : k;
    }
    return k;
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
