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

// DB: dbias is wanted too; without it the registers of its sums are free.
template <int G, int K, bool DG, bool DB>
__global__ __launch_bounds__(kThreads) void ns_bwd_kernel(NsBwdArgs a) {
  constexpr bool SUMS = DG || DB;
  __shared__ float sums[SUMS ? kThreads / G : 1][SUMS ? G * 8 : 1];
  const int gl = threadIdx.x % G, row0 = threadIdx.x / G;
  const int V = a.C / 8;
  const float root = sqrtf((float)a.C), inv_c = 1.0f / (float)a.C;
  Held<Bf16> gamma[K];
  float dg[DG ? K : 1][8], db[DB ? K : 1][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    gamma[k].v = u32x4_t{0, 0, 0, 0};
    if (gl + k * G < V) gamma[k].v = ((const u32x4_t*)a.gamma)[gl + k * G];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (DG) dg[k][j] = 0.0f;
      if (DB) db[k][j] = 0.0f;
    }
  }
  const long long step = (long long)gridDim.x * (kThreads / G);
  long long r = (long long)blockIdx.x * (kThreads / G) + row0;
  Held<Bf16> v[K], d[K];
  const auto load = [&](long long row) {
    const long long at = row * V + gl;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k].v = d[k].v = u32x4_t{0, 0, 0, 0};
      if (gl + k * G < V) {
        v[k].v = ((const u32x4_t*)a.value)[at + k * G];
        d[k].v = ((const u32x4_t*)a.dy)[at + k * G];
      }
    }
  };
  if (r < a.M) load(r);
  for (; r < a.M; r += step) {
    const long long at = r * V + gl;
    Held<Bf16> sk[K];
    if (a.dskip) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (gl + k * G < V) sk[k].v = ((const u32x4_t*)a.dskip)[at + k * G];
    }
    float n2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float x[8];
      v[k].get(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) n2 = fmaf(x[j], x[j], n2);
    }
    n2 = group_sum<G>(n2);
    const float norm = sqrtf(n2);
    const bool clamped = norm <= 1e-12f;             // and not fmaxf: a NaN stays
    const float s = root / (clamped ? 1e-12f : norm);
    float g[K][8], dot = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      // a vector's values step by step, so that no exponential or reciprocal
      // is waited for alone
      constexpr float kLog2e = 1.44269502162933349609375f;
      float e[8], gm[8], t[8], dy[8];
      v[k].get(e);
      gamma[k].get(gm);
      d[k].get(dy);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        e[j] *= s;
        g[k][j] = e[j] * gm[j];
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = __builtin_amdgcn_exp2f(g[k][j] * -kLog2e);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = __builtin_amdgcn_rcpf(1.0f + t[j]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float da = dy[j] * (t[j] * fmaf(g[k][j], 1.0f - t[j], 1.0f));
        if (DG) dg[k][j] = fmaf(da, e[j], dg[k][j]);
        g[k][j] = da * gm[j];
        dot = fmaf(g[k][j], e[j], dot);
      }
    }
    // g v / |v|^2 with g and v scaled: (g s)(v s) / (s |v|)^2, and s |v| = root
    dot = group_sum<G>(dot);
    const float back = clamped ? 0.0f : dot * inv_c * s;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float o[8], x[8], y[8];
      v[k].get(x);
      if (a.dskip) sk[k].get(y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = s * fmaf(-x[j], back, g[k][j]);
        if (a.dskip) o[j] += y[j];
        if (DB) db[k][j] += o[j];
      }
      Held<Bf16> out;
      out.put(o);
      if (gl + k * G < V) ((u32x4_t*)a.dvalue)[at + k * G] = out.v;
    }
    if (r + step < a.M) load(r + step);
  }
  if (SUMS) {
    float* out = a.partial + (long long)blockIdx.x * 2 * a.C;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (which ? !DB : !DG) continue;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          sums[row0][gl * 8 + j] = which ? db[DB ? k : 0][j] : dg[DG ? k : 0][j];
        __syncthreads();
        for (int i = threadIdx.x; i < G * 8 && k * G * 8 + i < a.C; i += kThreads) {
          float t = 0.0f;
          for (int q = 0; q < kThreads / G; ++q) t += sums[q][i];
          out[which * a.C + k * G * 8 + i] = t;
        }
      }
    }
  }
}

template <int G, int K>
void launch(const NsBwdArgs& a, hipStream_t s) {
  const dim3 grid(a.blocks), block(kThreads);
  if (a.dbias)
    hipLaunchKernelGGL((ns_bwd_kernel<G, K, true, true>), grid, block, 0, s, a);
  else if (a.dgamma)
    hipLaunchKernelGGL((ns_bwd_kernel<G, K, true, false>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((ns_bwd_kernel<G, K, false, false>), grid, block, 0, s, a);
}

// Lanes that share a row: the fewest (a power of two, at most a wave) whose
// three vectors each cover it; four only for the widest rows (their registers
// leave one wave per SIMD).
int lanes_per_row(int C) {
  const int V = C / 8;
  int g = 1;
  while (g < 64 && g * 3 < V) g *= 2;
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
  // lanes_per_row leaves no other pairs
#define CONV3D_NS_CASE(G)                       \
  case G:                                       \
    if (k == 2) launch<G, 2>(a, s);             \
    else launch<G, 3>(a, s);                    \
    break;
  switch (g) {
    case 1:
      if (k == 1) launch<1, 1>(a, s);
      else if (k == 2) launch<1, 2>(a, s);
      else launch<1, 3>(a, s);
      break;
    CONV3D_NS_CASE(2)
    CONV3D_NS_CASE(4)
    CONV3D_NS_CASE(8)
    CONV3D_NS_CASE(16)
    CONV3D_NS_CASE(32)
    default:
      if (k == 2) launch<64, 2>(a, s);
      else if (k == 3) launch<64, 3>(a, s);
      else launch<64, 4>(a, s);
  }
#undef CONV3D_NS_CASE
  if (a.dgamma || a.dbias)
    hipLaunchKernelGGL(column_sums_kernel, dim3((2 * a.C + kSumCols - 1) / kSumCols),
                       dim3(kSumThreads), 0, s, a.partial, a.blocks, a.C, a.dgamma, a.dbias);
  return (int)hipGetLastError();
}

}  // namespace conv3d
