// Backward pass of the channel L2 norm x sqrt(C) x gamma -> SiLU (the
// post-operations of conv3d_norm_silu and of the fused conv epilogue).
//
// For a pixel's channel row v (C values, the `value` of the forward pass),
// without the forward pass's intermediate roundings and with one at the end:
//   den = max(|v|, 1e-12), s = sqrt(C) / den, e = v s, a = e gamma, y = a sigmoid(a)
//   da = dy (sigmoid(a) + a sigmoid'(a)), g = da gamma s
//   dv = g - v (sum_c g v) / |v|^2 where |v| > 1e-12, else g   (+ dskip)
//   dgamma_c = sum over the rows of da e, dbias_c = of dv
//
// HBM-bound: value, dy (and dskip) are read once and dvalue is written once,
// the rows' sums stay in registers. G lanes (a power of two) share a row and
// hold K vectors of 8 channels each, so the two row sums (|v|^2, g v) are
// log2 G exchanges inside a wave and no barrier; a lane always holds the same
// channels, so gamma and the sums for dgamma and dbias stay in registers over
// all of a wave's rows. The sums of the rows of one work-group are joined in
// LDS and those of the work-groups by a second kernel, both in a fixed order.
#include <hip/hip_runtime.h>

#include "conv3d_device.h"
#include "conv3d_colsum.h"
#include "conv3d_elt.h"
#include "conv3d_train.h"

namespace conv3d {
namespace {

constexpr int kThreads = 256;

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

template <int G, int K, bool SUMS>
__global__ __launch_bounds__(kThreads) void ns_bwd_kernel(NsBwdArgs a) {
  typedef Pack<Bf16, 8> V8;
  __shared__ float sums[SUMS ? kThreads / G : 1][SUMS ? G * 8 : 1];
  const int gl = threadIdx.x % G, row0 = threadIdx.x / G;
  const int V = a.C / 8;
  const float root = sqrtf((float)a.C);
  float gamma[K][8], dg[K][8], db[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int cv = gl + k * G;
    if (cv < V) {
      unpack<Bf16, 8>(((const V8*)a.gamma)[cv], gamma[k]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) gamma[k][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[k][j] = db[k][j] = 0.0f;
  }
  const long long step = (long long)gridDim.x * (kThreads / G);
  for (long long r = (long long)blockIdx.x * (kThreads / G) + row0; r < a.M; r += step) {
    const long long at = r * V + gl;
    V8 pv[K], pd[K], ps[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (gl + k * G < V) {
        pv[k] = ((const V8*)a.value)[at + k * G];
        pd[k] = ((const V8*)a.dy)[at + k * G];
        if (a.dskip) ps[k] = ((const V8*)a.dskip)[at + k * G];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) pv[k].v[j] = pd[k].v[j] = 0;
      }
    }
    float v[K][8], g[K][8], n2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unpack<Bf16, 8>(pv[k], v[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) n2 = fmaf(v[k][j], v[k][j], n2);
    }
    n2 = group_sum<G>(n2);
    const float norm = sqrtf(n2);
    const bool clamped = norm <= 1e-12f;             // and not fmaxf: a NaN stays
    const float s = root / (clamped ? 1e-12f : norm);
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float d[8];
      unpack<Bf16, 8>(pd[k], d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = v[k][j] * s, act = e * gamma[k][j];
        const float da = d[j] * silu_slope<false>(act);
        if (SUMS) dg[k][j] = fmaf(da, e, dg[k][j]);
        g[k][j] = da * gamma[k][j];
        dot = fmaf(g[k][j], e, dot);
      }
    }
    // g v / |v|^2 with g and v scaled: (g s)(v s) / (s |v|)^2, and s |v| = root
    dot = group_sum<G>(dot);
    const float back = clamped ? 0.0f : dot / (float)a.C;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (gl + k * G >= V) continue;
      float o[8], sk[8];
      if (a.dskip) unpack<Bf16, 8>(ps[k], sk);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = s * (g[k][j] - v[k][j] * s * back);
        if (a.dskip) o[j] += sk[j];
        if (SUMS) db[k][j] += o[j];
      }
      ((V8*)a.dvalue)[at + k * G] = pack<Bf16, 8>(o);
    }
  }
  if (SUMS) {
    float* out = a.partial + (long long)blockIdx.x * 2 * a.C;
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[row0][gl * 8 + j] = which ? db[k][j] : dg[k][j];
        __syncthreads();
        const int c = k * G * 8 + threadIdx.x;
        if (threadIdx.x < G * 8 && c < a.C) {
          float t = 0.0f;
          for (int i = 0; i < kThreads / G; ++i) t += sums[i][threadIdx.x];
          out[which * a.C + c] = t;
        }
        if (G * 8 > kThreads && threadIdx.x + kThreads < G * 8 && c + kThreads < a.C) {
          float t = 0.0f;
          for (int i = 0; i < kThreads / G; ++i) t += sums[i][threadIdx.x + kThreads];
          out[which * a.C + c + kThreads] = t;
        }
      }
  }
}

template <int G, int K>
void launch(const NsBwdArgs& a, hipStream_t s) {
  if (a.dgamma || a.dbias)
    hipLaunchKernelGGL((ns_bwd_kernel<G, K, true>), dim3(a.blocks), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((ns_bwd_kernel<G, K, false>), dim3(a.blocks), dim3(kThreads), 0, s, a);
}

// Lanes that share a row: the fewest (a power of two) whose K <= 4 vectors
// each cover it.
int lanes_per_row(int C) {
  const int V = C / 8;
  int g = 1;
  while (g * 4 < V) g *= 2;
  return g;
}

}  // namespace

int ns_bwd_blocks(long long M, int C) {
  const long long rows = kThreads / lanes_per_row(C);       // of a work-group's pass
  const long long passes = (M + rows - 1) / rows;
  return (int)(passes < 1024 ? passes : 1024);
}

int launch_ns_bwd(const NsBwdArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  const int V = a.C / 8, g = lanes_per_row(a.C), k = (V + g - 1) / g;
#define CONV3D_NS_CASE(G)                       \
  case G:                                       \
    if (k == 1) launch<G, 1>(a, s);             \
    else if (k == 2) launch<G, 2>(a, s);        \
    else if (k == 3) launch<G, 3>(a, s);        \
    else launch<G, 4>(a, s);                    \
    break;
  switch (g) {
    CONV3D_NS_CASE(1)
    CONV3D_NS_CASE(2)
    CONV3D_NS_CASE(4)
    CONV3D_NS_CASE(8)
    CONV3D_NS_CASE(16)
    CONV3D_NS_CASE(32)
    CONV3D_NS_CASE(64)
  }
#undef CONV3D_NS_CASE
  if (a.dgamma || a.dbias)
    hipLaunchKernelGGL(column_sums_kernel, dim3((2 * a.C + kSumCols - 1) / kSumCols),
                       dim3(kSumThreads), 0, s, a.partial, a.blocks, a.C, a.dgamma, a.dbias);
  return (int)hipGetLastError();
}

}  // namespace conv3d
