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

// 16 bytes of elements as they are kept in registers, four of them: the
// compiler would give every 16-bit element of a Pack a register of its own.
template <class T>
struct Held {
  static constexpr int VEC = 16 / sizeof(typename T::store);
  u32x4_t v;
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
    if constexpr (VEC == 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = __builtin_bit_cast(float, (unsigned)v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = T::get((typename T::store)(v[j] & 0xffffu));
        f[2 * j + 1] = T::get((typename T::store)(v[j] >> 16));
      }
    }
  }
  __device__ __forceinline__ void put(const float (&f)[VEC]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (VEC == 4) v[j] = __builtin_bit_cast(unsigned, f[j]);
      else v[j] = (unsigned)T::put(f[2 * j]) | ((unsigned)T::put(f[2 * j + 1]) << 16);
    }
  }
};
template <>
__device__ __forceinline__ void Held<Bf16>::get(float (&f)[8]) const {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf_lo(v[j]);
    f[2 * j + 1] = bf_hi(v[j]);
  }
}
template <>
__device__ __forceinline__ void Held<Bf16>::put(const float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = pack2(f[2 * j], f[2 * j + 1]);
}

// e^-a. 16-bit results: t = 2^(-a log2 e) by the hardware
// exponential; it overflows to infinity below a = -88, where 1 / (1 + t) = 0 is
// the rounded value anyway. fp32 results (EXACT): the rounding of a log2 e is
// made good by a second product, and only e^-|a| is formed, so that 1 - sig
// needs no difference. A NaN stays one only where it is multiplied with: here
// the fp32 form makes it 0, and both uses below multiply by the argument.
template <bool EXACT>
__device__ __forceinline__ float exp_neg(float v) {
  constexpr float kLog2e = 1.44269502162933349609375f;
  if (!EXACT) return __builtin_amdgcn_exp2f(-v * kLog2e);
  constexpr float kLog2eLo = 1.925963033500011e-08f;   // log2(e) - kLog2e
  constexpr float kLn2 = 0.693147182464599609375f;
  const float m = fminf(v, 256.0f);                    // t is 0 there, and no infinity meets 0
  const float p = m * kLog2e;
  const float t = __builtin_amdgcn_exp2f(-p);
  const float r = __builtin_fmaf(m, kLog2eLo, __builtin_fmaf(m, kLog2e, -p));
  return __builtin_fmaf(t, -r * kLn2, t);
}

// a sigmoid(a).
template <bool EXACT>
__device__ __forceinline__ float silu_of(float a) {
  if (!EXACT) return a * __builtin_amdgcn_rcpf(1.0f + exp_neg<false>(a));
  const float t = exp_neg<true>(fabsf(a));
  const float q = __builtin_amdgcn_rcpf(1.0f + t);
  return a * (a >= 0.0f ? q : t * q);
}

// Its derivative sigmoid(a) (1 + a (1 - sigmoid(a))).
template <bool EXACT>
__device__ __forceinline__ float silu_slope(float a) {
  if (!EXACT) {
    const float sig = __builtin_amdgcn_rcpf(1.0f + exp_neg<false>(a));
    return sig * __builtin_fmaf(a, 1.0f - sig, 1.0f);
  }
  const float t = exp_neg<true>(fabsf(a));
  const float q = __builtin_amdgcn_rcpf(1.0f + t);
  return __builtin_fmaf(a, t * q * q, a >= 0.0f ? q : t * q);
}

}  // namespace conv3d
