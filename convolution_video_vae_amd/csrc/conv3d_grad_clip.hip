// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum over all tensors and elements of g^2), or max |g|
//   coef = min(1, max_norm / (norm + 1e-6)), a NaN norm gives a NaN
//   out  = g coef, rounded once to out's type
//
// HBM-bound: the norm pass reads every gradient once, the clip pass reads it
// again (no value can be scaled before the last one is summed) and writes it.
// In place and with coef = 1 the clip pass reads and writes nothing. Results
// that would fill half of the memory-side cache and more are stored past it:
// else their write-back slows the next norm pass, and the gradients that the
// clip pass finds there are pushed out (167 M bf16 gradients into fp32: 278 us,
// so 241 us).
//
// The tensors' addresses travel as kernel arguments, at most kGradItems per
// launch: no table is copied to the device, so a captured call needs no host
// memory afterwards. Work-groups are dealt to the tensors by a prefix of
// block counts, found by bisection. Squares are formed and summed in fp64
// (an fp32 square leaves the range from |g| > 1.8e19 and < 1e-23); each
// work-group leaves one partial, and every work-group of the clip pass adds
// all of them in the same fixed order, so no launch stands between the two
// passes and the result does not depend on the order of work-groups. Every
// tensor leaves a partial, and that work grows with their square: of many, one
// work-group adds them (in that order, to the same value) between the passes.
#include <hip/hip_runtime.h>

#include "conv3d_device.h"
#include "conv3d_elt.h"
#include "conv3d_train.h"

namespace conv3d {
namespace {

constexpr int kThreads = 256;

// Vectors of VEC elements at any element's alignment (a tensor may start
// anywhere in a larger buffer).
template <class T, int VEC>
struct __attribute__((packed, aligned(sizeof(typename T::store)))) Loose {
  typename T::store v[VEC];
};

__device__ __forceinline__ int find_item(const GradBatch& b, int block) {
  int lo = 0, hi = b.count - 1;         // the last item whose first block is <= block
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.item[mid].first <= block) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// |g| or g^2 joined into acc; a NaN stays.
template <bool INF>
__device__ __forceinline__ double join(double acc, float v) {
  if (INF) {
    const double m = fabsf(v);
    return (m > acc || m != m) ? m : acc;
  }
  return fma((double)v, (double)v, acc);
}
template <bool INF>
__device__ __forceinline__ double merge(double p, double q) {
  if (INF) return (q > p || q != q) ? q : p;
  return p + q;
}

// Over the work-group, in lane and wave order; every thread gets the result.
template <bool INF>
__device__ __forceinline__ double block_merge(double v) {
  __shared__ double w[kThreads / 64];
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = merge<INF>(v, __shfl_xor(v, m));
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = v;
  __syncthreads();
  v = w[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) v = merge<INF>(v, w[i]);
  return v;
}

template <class T, bool INF>
__device__ __forceinline__ double sum_range(const void* src, long long at, int n) {
  typedef typename T::store E;
  constexpr int VEC = 16 / sizeof(E), U = 8;
  typedef Loose<T, VEC> L;
  const E* p = (const E*)src + at;
  const int nv = n / VEC;
  double acc = 0.0;
  int i = threadIdx.x;
  for (; i + (U - 1) * kThreads < nv; i += U * kThreads) {
    L v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = *(const L*)(p + (long long)(i + k * kThreads) * VEC);
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc = join<INF>(acc, T::get(v[k].v[j]));
  }
  for (; i < nv; i += kThreads) {
    const L v = *(const L*)(p + (long long)i * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc = join<INF>(acc, T::get(v.v[j]));
  }
  const int e = nv * VEC + (int)threadIdx.x;
  if (e < n) acc = join<INF>(acc, T::get(p[e]));    // fewer than VEC are left
  return acc;
}

template <bool INF>
__global__ __launch_bounds__(kThreads) void grad_partials_kernel(GradBatch b) {
  const int i = find_item(b, blockIdx.x);
  const long long at = (long long)((int)blockIdx.x - b.item[i].first) * b.chunk;
  const int n = (int)min((long long)b.chunk, b.item[i].numel - at);
  const void* src = b.item[i].src;
  const int dtype = b.item[i].dtype;
  double acc;
  if (dtype == ELT_BF16) acc = sum_range<Bf16, INF>(src, at, n);
  else if (dtype == ELT_FP16) acc = sum_range<Fp16, INF>(src, at, n);
  else acc = sum_range<Fp32, INF>(src, at, n);
  acc = block_merge<INF>(acc);
  if (threadIdx.x == 0) b.partial[blockIdx.x] = acc;
}

template <bool INF>
__device__ __forceinline__ double join_partials(const GradBatch& b) {
  double acc = 0.0;
  for (int i = threadIdx.x; i < b.partials; i += kThreads) acc = merge<INF>(acc, b.all[i]);
  return block_merge<INF>(acc);
}
template <bool INF>
__device__ __forceinline__ double norm_of(double join) {
  return INF ? join : sqrt(join);
}

template <bool INF>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(GradBatch b) {
  const double join = join_partials<INF>(b);
  if (threadIdx.x) return;
  if (b.join) *b.join = join;
  *b.norm = (float)norm_of<INF>(join);
}

// A lane's vector of results; STREAM: past the caches (16 bytes, or 8 where the
// gradients are the wider type). Alignment is an element's, as for Loose.
template <class O, int VEC, bool STREAM>
__device__ __forceinline__ void store_scaled(typename O::store* q, const Loose<O, VEC>& o) {
  typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
  typedef u32x4_t loose16_t __attribute__((aligned(2)));
  typedef u32x2_t loose8_t __attribute__((aligned(2)));
  if constexpr (STREAM && sizeof(o) == 16) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, o), (loose16_t*)q);
  } else if constexpr (STREAM && sizeof(o) == 8) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x2_t, o), (loose8_t*)q);
  } else {
    *(Loose<O, VEC>*)q = o;
  }
}

template <class T, class O, bool STREAM>
__device__ __forceinline__ void scale_range(const void* src, void* dst, long long at, int n,
                                            float coef) {
  typedef typename T::store E;
  typedef typename O::store F;
  // 16 bytes of the wider type per lane, so that a wave's loads and stores are
  // both without gaps
  constexpr int VEC = 16 / (sizeof(E) > sizeof(F) ? sizeof(E) : sizeof(F)), U = 8;
  typedef Loose<T, VEC> L;
  typedef Loose<O, VEC> S;
  const E* p = (const E*)src + at;
  F* q = (F*)dst + at;
  const int nv = n / VEC;
  int i = threadIdx.x;
  for (; i + (U - 1) * kThreads < nv; i += U * kThreads) {
    L v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = *(const L*)(p + (long long)(i + k * kThreads) * VEC);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      S o;
#pragma unroll
      for (int j = 0; j < VEC; ++j) o.v[j] = O::put(T::get(v[k].v[j]) * coef);
      store_scaled<O, VEC, STREAM>(q + (long long)(i + k * kThreads) * VEC, o);
    }
  }
  for (; i < nv; i += kThreads) {
    const L v = *(const L*)(p + (long long)i * VEC);
    S o;
#pragma unroll
    for (int j = 0; j < VEC; ++j) o.v[j] = O::put(T::get(v.v[j]) * coef);
    *(S*)(q + (long long)i * VEC) = o;
  }
  const int e = nv * VEC + (int)threadIdx.x;
  if (e < n) q[e] = O::put(T::get(p[e]) * coef);
}

template <class T, bool STREAM>
__device__ __forceinline__ void scale_to(const void* src, void* dst, int out, long long at, int n,
                                         float coef) {
  if (out == ELT_BF16) scale_range<T, Bf16, STREAM>(src, dst, at, n, coef);
  else if (out == ELT_FP16) scale_range<T, Fp16, STREAM>(src, dst, at, n, coef);
  else scale_range<T, Fp32, STREAM>(src, dst, at, n, coef);
}

template <bool INF, bool STREAM>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradBatch b) {
  const double norm = norm_of<INF>(join_partials<INF>(b));
  if (b.norm && blockIdx.x == 0 && threadIdx.x == 0) *b.norm = (float)norm;
  const double c = (double)b.max_norm / (norm + 1e-6);
  const float coef = c > 1.0 ? 1.0f : (float)c;      // a NaN is not above 1
  // from the last block back: what the norm pass read last is still in the
  // memory-side cache
  const int block = gridDim.x - 1 - blockIdx.x;
  const int i = find_item(b, block);
  const void* src = b.item[i].src;
  void* dst = b.item[i].dst;
  const int dtype = b.item[i].dtype, out = b.item[i].out_dtype;
  if (coef == 1.0f && src == dst) return;            // in place, and nothing changes
  const long long at = (long long)(block - b.item[i].first) * b.chunk;
  const int n = (int)min((long long)b.chunk, b.item[i].numel - at);
  if (dtype == ELT_BF16) scale_to<Bf16, STREAM>(src, dst, out, at, n, coef);
  else if (dtype == ELT_FP16) scale_to<Fp16, STREAM>(src, dst, out, at, n, coef);
  else scale_to<Fp32, STREAM>(src, dst, out, at, n, coef);
}

}  // namespace

int launch_grad_partials(const GradBatch& b, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  if (b.inf)
    hipLaunchKernelGGL(grad_partials_kernel<true>, dim3(b.blocks), dim3(kThreads), 0, s, b);
  else
    hipLaunchKernelGGL(grad_partials_kernel<false>, dim3(b.blocks), dim3(kThreads), 0, s, b);
  return (int)hipGetLastError();
}

int launch_grad_norm(const GradBatch& b, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  if (b.inf) hipLaunchKernelGGL(grad_norm_kernel<true>, dim3(1), dim3(kThreads), 0, s, b);
  else hipLaunchKernelGGL(grad_norm_kernel<false>, dim3(1), dim3(kThreads), 0, s, b);
  return (int)hipGetLastError();
}

int launch_grad_scale(const GradBatch& b, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  const dim3 grid(b.blocks), block(kThreads);
  if (b.inf && b.stream)
    hipLaunchKernelGGL((grad_scale_kernel<true, true>), grid, block, 0, s, b);
  else if (b.inf)
    hipLaunchKernelGGL((grad_scale_kernel<true, false>), grid, block, 0, s, b);
  else if (b.stream)
    hipLaunchKernelGGL((grad_scale_kernel<false, true>), grid, block, 0, s, b);
  else
    hipLaunchKernelGGL((grad_scale_kernel<false, false>), grid, block, 0, s, b);
  return (int)hipGetLastError();
}

}  // namespace conv3d
