// Element types of the training-side kernels: storage, conversion to and
// from fp32 (round to nearest even) and vectors of VEC elements.
#pragma once

#include <hip/hip_runtime.h>

#include "conv3d_device.h"

namespace conv3d {

struct Bf16 {
  typedef uint16_t store;
  static constexpr bool kWide = false;
  static __device__ __forceinline__ float get(store v) { return bf2f(v); }
  static __device__ __forceinline__ store put(float f) { return f2bf(f); }
};
struct Fp16 {
  typedef uint16_t store;
  static constexpr bool kWide = false;
  static __device__ __forceinline__ float get(store v) {
    return (float)__builtin_bit_cast(_Float16, v);
  }
  static __device__ __forceinline__ store put(float f) {
    return __builtin_bit_cast(uint16_t, (_Float16)f);
  }
};
struct Fp32 {
  typedef float store;
  static constexpr bool kWide = true;
  static __device__ __forceinline__ float get(store v) { return v; }
  static __device__ __forceinline__ store put(float f) { return f; }
};

// VEC elements as one aligned piece of memory.
template <class T, int VEC>
struct alignas(VEC * sizeof(typename T::store)) Pack {
  typename T::store v[VEC];
};

template <class T, int VEC>
__device__ __forceinline__ void unpack(const Pack<T, VEC>& p, float (&f)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) f[j] = T::get(p.v[j]);
}
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> pack(const float (&f)[VEC]) {
  Pack<T, VEC> p;
#pragma unroll
  for (int j = 0; j < VEC; ++j) p.v[j] = T::put(f[j]);
  return p;
}

// The parts of the logistic function for a: with t = e^-|a| (<= 1, nothing
// overflows) and q = 1 / (1 + t), sigmoid(a) is q for a >= 0 and t q below,
// and its slope is t q^2. e^-|a| is 2^-(|a| log2 e); with EXACT the rounding
// of that product is made good (fp32 results; below the rounding of 16-bit
// ones). |a| is capped where t is zero anyway, so no infinity meets its
// negative; a NaN goes through the callers' products with a.
template <bool EXACT>
__device__ __forceinline__ void logistic(float a, float& sig, float& slope) {
  constexpr float kLog2e = 1.44269502162933349609375f;
  constexpr float kLog2eLo = 1.925963033500011e-08f;   // log2(e) - kLog2e
  constexpr float kLn2 = 0.693147182464599609375f;
  const float m = fminf(fabsf(a), 256.0f);
  const float p = m * kLog2e;
  float t = __builtin_amdgcn_exp2f(-p);
  if (EXACT) {
    const float r = __builtin_fmaf(m, kLog2eLo, __builtin_fmaf(m, kLog2e, -p));
    t = __builtin_fmaf(t, -r * kLn2, t);
  }
  const float q = __builtin_amdgcn_rcpf(1.0f + t);
  sig = a >= 0.0f ? q : t * q;
  slope = t * q * q;
}

}  // namespace conv3d
