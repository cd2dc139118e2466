// Channels-last GroupNorm (+ SiLU) for training: the forward pass that keeps
// its statistics, and the backward pass.
//
// Over a unit (one frame, or one sample) of P pixels and a group of K
// consecutive channels, N = P K values, with one rounding at the end:
//   forward   mean = sum x / N, rstd = 1 / sqrt(sum (x - mean)^2 / N + eps)
//             h = (x - mean) rstd, a = h gamma_c + beta_c, y = a or a sigmoid(a)
//   backward  da = dy, or dy (sigmoid(a) + a sigmoid'(a))
//             A_c = sum over the unit's pixels of da, B_c = of da h
//             c1 = sum over the group of gamma_c A_c / N, c2 = of gamma_c B_c / N
//             dx = rstd (gamma_c da - c1 - h c2)
//             dbeta_c = sum over the units of A_c, dgamma_c = of B_c
//
// Both passes read the activations twice: once for the sums, once for the
// result (the sums of a unit are not known before its last pixel is read).
//   sums      one work-group per (unit, chunk of pixels), per-thread sums in
//             fp32 over at most a chunk's share, joined in fp64 in a fixed
//             order, one (first, second) pair per channel and chunk
//   finalize  chunk pairs in a fixed order -> the group's statistics, or the
//             unit's channel sums and the group's c1, c2
//   result    elementwise, from the last chunk back: what the sums pass read
//             last is still in the memory-side cache. Results that would fill
//             half of it and more are stored past it ([1,17,256,256,128] bf16
//             with statistics over the clip, forward 192 -> 162 us, backward
//             307 -> 287 us)
//   params    dgamma, dbeta from the units' channel sums, in unit order
// No atomics: results do not depend on the order of work-groups.
//
// Variance: each thread shifts its channels by the first value it meets, so
// its fp32 sums hold the spread and not the mean. The sums that it leaves are
// about ref, the group's first value (x - ref = shift - ref + d, in fp64): about
// zero, a constant group of 30000 would have a variance of 1e-7 instead of 0,
// which is 1e-2 of eps.
//
// Vectors: a thread always holds the same VEC elements of a row, so its
// channels' constants stay in registers. A row is one pixel where VEC
// divides C, and otherwise, in dense tensors, the fewest pixels that are a
// whole number of vectors (3 channels and 8-element vectors: 8 pixels).
#include <hip/hip_runtime.h>

#include "conv3d_device.h"
#include "conv3d_elt.h"
#include "conv3d_gn_device.h"
#include "conv3d_train.h"

namespace conv3d {
namespace {

constexpr int kThreads = 256;

// How a launch lays the unit's rows over its threads.
struct Rows {
  long long Q;          // rows per unit
  long long chunk_q;    // rows per chunk
  int sp;               // pixels per row
  int V;                // vectors per row
  int Vt, tiles;        // vectors of one channel tile; tiles (1 unless V > kThreads)
  int ppi;              // rows per pass of a work-group
};

struct Lane {
  int cv, pl;
  bool active;
};

__device__ __forceinline__ Lane lane_of(const Rows& r) {
  Lane l;
  const int t = threadIdx.x;
  l.pl = t / r.Vt;
  l.cv = t - l.pl * r.Vt + blockIdx.y * r.Vt;
  l.active = l.pl < r.ppi && l.cv < r.V;
  return l;
}

// Channel of element j of vector cv.
template <int VEC>
__device__ __forceinline__ int channel(const GnTrainArgs& a, int cv, int j) {
  return (cv * VEC + j) % a.C;
}

// One lane's rows q0, q0 + ppi, ... below q1, U at a time: f(row, k) loads row
// into slot k, g(row, k) uses slot k.
template <int U, class Load, class Use>
__device__ __forceinline__ void each_row(long long q0, long long q1, int ppi, Load load, Use use) {
  if (q0 >= q1) return;
  const int n = (int)((q1 - q0 + ppi - 1) / ppi);   // a chunk holds below 2^31 rows
  int i = 0;
  for (; i + U <= n; i += U) {
    const long long q = q0 + (long long)i * ppi;
#pragma unroll
    for (int k = 0; k < U; ++k) load(q + (long long)k * ppi, k);
#pragma unroll
    for (int k = 0; k < U; ++k) use(q + (long long)k * ppi, k);
  }
  const long long q = q0 + (long long)i * ppi;
#pragma unroll
  for (int k = 0; k < U; ++k)
    if (i + k < n) load(q + (long long)k * ppi, k);
#pragma unroll
  for (int k = 0; k < U; ++k)
    if (i + k < n) use(q + (long long)k * ppi, k);
}

// Joins the work-group's (v1, v2) pairs per channel over its rows' lanes and
// the row's pixels, in that order, and writes them to `out` [C][2].
template <int VEC>
__device__ __forceinline__ void join_channels(const GnTrainArgs& a, const Rows& r, const Lane& l,
                                              const double (&v1)[VEC], const double (&v2)[VEC],
                                              double* out) {
  __shared__ double r1[kThreads * VEC], r2[kThreads * VEC];
  if (l.active) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      r1[threadIdx.x * VEC + j] = v1[j];
      r2[threadIdx.x * VEC + j] = v2[j];
    }
  }
  __syncthreads();
  const int width = r.Vt * VEC;                       // elements of one lane row
  const int c0 = blockIdx.y * width;
  const int nc = r.tiles == 1 ? a.C : min(width, a.C - c0);
  for (int c = threadIdx.x; c < nc; c += kThreads) {
    double t1 = 0.0, t2 = 0.0;
    for (int pl = 0; pl < r.ppi; ++pl)
      for (int s = 0; s < r.sp; ++s) {
        t1 += r1[pl * width + s * a.C + c];
        t2 += r2[pl * width + s * a.C + c];
      }
    out[(c0 + c) * 2] = t1;
    out[(c0 + c) * 2 + 1] = t2;
  }
}

// A vector of results; STREAM (16-byte vectors): past the caches.
template <bool STREAM, class T, int VEC>
__device__ __forceinline__ void store_pack(void* p, const Pack<T, VEC>& v) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), (u32x4_t*)p);
  else
    *(Pack<T, VEC>*)p = v;
}

// The first value of a unit and group.
template <class T>
__device__ __forceinline__ float group_ref(const GnTrainArgs& a, int u, int g) {
  return T::get(((const typename T::store*)a.x)[(long long)u * a.P * a.x_pitch + g * a.cpg]);
}

template <class T, int VEC>
__global__ __launch_bounds__(kThreads) void gn_train_stats_kernel(GnTrainArgs a, Rows r) {
  typedef typename T::store E;
  constexpr int U = 8;
  const int u = blockIdx.x / a.chunks, k = blockIdx.x - u * a.chunks;
  const Lane l = lane_of(r);
  double t1[VEC], t2[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) t1[j] = t2[j] = 0.0;
  if (l.active) {
    const long long pitch = r.sp * a.x_pitch;
    const E* x = (const E*)a.x + (long long)u * a.P * a.x_pitch + l.cv * VEC;
    const long long q0 = k * r.chunk_q + l.pl, q1 = min(r.Q, (k + 1) * r.chunk_q);
    float ref[VEC], sh[VEC], s1[VEC], s2[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      ref[j] = group_ref<T>(a, u, channel<VEC>(a, l.cv, j) / a.cpg);
      sh[j] = s1[j] = s2[j] = 0.0f;
    }
    if (q0 < q1) unpack<T, VEC>(*(const Pack<T, VEC>*)(x + q0 * pitch), sh);
    Pack<T, VEC> v[U];
    each_row<U>(
        q0, q1, r.ppi,
        [&](long long q, int i) { v[i] = *(const Pack<T, VEC>*)(x + q * pitch); },
        [&](long long, int i) {
          float f[VEC];
          unpack<T, VEC>(v[i], f);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float d = f[j] - sh[j];
            s1[j] += d;
            s2[j] = fmaf(d, d, s2[j]);
          }
        });
    const double n = q0 < q1 ? (double)((q1 - q0 + r.ppi - 1) / r.ppi) : 0.0;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const double s = (double)sh[j] - (double)ref[j];
      t1[j] = n * s + s1[j];
      t2[j] = n * s * s + 2.0 * s * s1[j] + s2[j];
    }
  }
  join_channels<VEC>(a, r, l, t1, t2, a.partial + (long long)blockIdx.x * a.C * 2);
}

// Sums two values over the work-group, in lane and wave order.
__device__ __forceinline__ void block_sum(double& v1, double& v2) {
  __shared__ double w1[kThreads / 64], w2[kThreads / 64];
  v1 = wave_sum(v1);
  v2 = wave_sum(v2);
  if ((threadIdx.x & 63) == 0) {
    w1[threadIdx.x >> 6] = v1;
    w2[threadIdx.x >> 6] = v2;
  }
  __syncthreads();
  v1 = v2 = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    v1 += w1[w];
    v2 += w2[w];
  }
}

// One work-group per (unit, group).
template <class T>
__global__ __launch_bounds__(kThreads) void gn_train_stats_finalize_kernel(GnTrainArgs a) {
  const int u = blockIdx.x / a.G, g = blockIdx.x - u * a.G;
  const float ref = group_ref<T>(a, u, g);
  const double* part = a.partial + ((long long)u * a.chunks * a.C + g * a.cpg) * 2;
  double s1 = 0.0, s2 = 0.0;
  const long long n = (long long)a.chunks * a.cpg;
  for (long long i = threadIdx.x; i < n; i += kThreads) {
    const long long k = i / a.cpg, c = i - k * a.cpg;
    s1 += part[(k * a.C + c) * 2];
    s2 += part[(k * a.C + c) * 2 + 1];
  }
  block_sum(s1, s2);
  if (threadIdx.x == 0) {
    const double N = (double)a.P * a.cpg;
    const double off = s1 / N;
    double var = s2 / N - off * off;
    if (var < 0.0) var = 0.0;                   // and not fmax: a NaN stays
    a.stats[(long long)blockIdx.x * 2] = (float)((double)ref + off);
    a.stats[(long long)blockIdx.x * 2 + 1] = (float)(1.0 / sqrt(var + (double)a.eps));
  }
}

template <class T, int VEC, bool SILU, bool STREAM>
__global__ __launch_bounds__(kThreads) void gn_train_apply_kernel(GnTrainArgs a, Rows r) {
  typedef typename T::store E;
  constexpr int U = 8;
  const int item = gridDim.x - 1 - blockIdx.x;
  const int u = item / a.chunks, k = item - u * a.chunks;
  const Lane l = lane_of(r);
  if (!l.active) return;
  float mean[VEC], scale[VEC], beta[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int c = channel<VEC>(a, l.cv, j);
    const float* st = a.stats + ((long long)u * a.G + c / a.cpg) * 2;
    mean[j] = st[0];
    scale[j] = st[1] * a.gamma[c];
    beta[j] = a.beta[c];
  }
  const long long xp = r.sp * a.x_pitch, yp = r.sp * a.out_pitch;
  const E* x = (const E*)a.x + (long long)u * a.P * a.x_pitch + l.cv * VEC;
  E* y = (E*)a.out + (long long)u * a.P * a.out_pitch + l.cv * VEC;
  Pack<T, VEC> v[U];
  each_row<U>(
      k * r.chunk_q + l.pl, min(r.Q, (k + 1) * r.chunk_q), r.ppi,
      [&](long long q, int i) { v[i] = *(const Pack<T, VEC>*)(x + q * xp); },
      [&](long long q, int i) {
        float f[VEC];
        unpack<T, VEC>(v[i], f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          f[j] = fmaf(f[j] - mean[j], scale[j], beta[j]);
          if (SILU) f[j] = silu_of<T::kWide>(f[j]);
        }
        store_pack<STREAM>(y + q * yp, pack<T, VEC>(f));
      });
}

// The constants of a thread's channels, and da and h of one vector.
template <class T, int VEC, bool SILU>
struct BwdLane {
  float mean[VEC], rstd[VEC], gamma[VEC], beta[VEC];
  __device__ __forceinline__ void init(const GnTrainArgs& a, int u, int cv) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = channel<VEC>(a, cv, j);
      const float* st = a.stats + ((long long)u * a.G + c / a.cpg) * 2;
      mean[j] = st[0];
      rstd[j] = st[1];
      gamma[j] = a.gamma[c];
      beta[j] = a.beta[c];
    }
  }
  __device__ __forceinline__ void value(int j, float x, float dy, float& h, float& da) const {
    h = (x - mean[j]) * rstd[j];
    da = SILU ? dy * silu_slope<T::kWide>(fmaf(h, gamma[j], beta[j])) : dy;
  }
};

template <class T, int VEC, bool SILU>
__global__ __launch_bounds__(kThreads) void gn_train_bwd_sums_kernel(GnTrainArgs a, Rows r) {
  typedef typename T::store E;
  constexpr int U = 4;
  const int u = blockIdx.x / a.chunks, k = blockIdx.x - u * a.chunks;
  const Lane l = lane_of(r);
  double t1[VEC], t2[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) t1[j] = t2[j] = 0.0;
  if (l.active) {
    BwdLane<T, VEC, SILU> b;
    b.init(a, u, l.cv);
    const long long xp = r.sp * a.x_pitch, dp = r.sp * a.dy_pitch;
    const E* x = (const E*)a.x + (long long)u * a.P * a.x_pitch + l.cv * VEC;
    const E* dy = (const E*)a.dy + (long long)u * a.P * a.dy_pitch + l.cv * VEC;
    float s1[VEC], s2[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s1[j] = s2[j] = 0.0f;
    Pack<T, VEC> vx[U], vd[U];
    each_row<U>(
        k * r.chunk_q + l.pl, min(r.Q, (k + 1) * r.chunk_q), r.ppi,
        [&](long long q, int i) {
          vx[i] = *(const Pack<T, VEC>*)(x + q * xp);
          vd[i] = *(const Pack<T, VEC>*)(dy + q * dp);
        },
        [&](long long, int i) {
          float f[VEC], d[VEC];
          unpack<T, VEC>(vx[i], f);
          unpack<T, VEC>(vd[i], d);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            float h, da;
            b.value(j, f[j], d[j], h, da);
            s1[j] += da;
            s2[j] = fmaf(da, h, s2[j]);
          }
        });
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      t1[j] = s1[j];
      t2[j] = s2[j];
    }
  }
  join_channels<VEC>(a, r, l, t1, t2, a.partial + (long long)blockIdx.x * a.C * 2);
}

// One work-group per (unit, group): a wave takes every fourth channel of the
// group and sums its chunks; the work-group then joins gamma_c A_c and
// gamma_c B_c.
__global__ __launch_bounds__(kThreads) void gn_train_bwd_finalize_kernel(GnTrainArgs a) {
  const int u = blockIdx.x / a.G, g = blockIdx.x - u * a.G;
  const int lane = threadIdx.x & 63;
  double d1 = 0.0, d2 = 0.0;
  for (int i = threadIdx.x >> 6; i < a.cpg; i += kThreads / 64) {
    const int c = g * a.cpg + i;
    const double* part = a.partial + ((long long)u * a.chunks * a.C + c) * 2;
    double s1 = 0.0, s2 = 0.0;
    for (int k = lane; k < a.chunks; k += 64) {
      s1 += part[(long long)k * a.C * 2];
      s2 += part[(long long)k * a.C * 2 + 1];
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if (lane == 0) {
      a.chan[((long long)u * a.C + c) * 2] = s1;
      a.chan[((long long)u * a.C + c) * 2 + 1] = s2;
      d1 += a.gamma[c] * s1;
      d2 += a.gamma[c] * s2;
    }
  }
  block_sum(d1, d2);
  if (threadIdx.x == 0) {
    const double N = (double)a.P * a.cpg;
    a.coef[(long long)blockIdx.x * 2] = (float)(d1 / N);
    a.coef[(long long)blockIdx.x * 2 + 1] = (float)(d2 / N);
  }
}

template <class T, int VEC, bool SILU, bool STREAM>
__global__ __launch_bounds__(kThreads) void gn_train_bwd_apply_kernel(GnTrainArgs a, Rows r) {
  typedef typename T::store E;
  constexpr int U = 4;
  const int item = gridDim.x - 1 - blockIdx.x;
  const int u = item / a.chunks, k = item - u * a.chunks;
  const Lane l = lane_of(r);
  if (!l.active) return;
  BwdLane<T, VEC, SILU> b;
  b.init(a, u, l.cv);
  float c1[VEC], c2[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const float* co = a.coef + ((long long)u * a.G + channel<VEC>(a, l.cv, j) / a.cpg) * 2;
    c1[j] = co[0];
    c2[j] = co[1];
  }
  const long long xp = r.sp * a.x_pitch, dp = r.sp * a.dy_pitch, op = r.sp * a.out_pitch;
  const E* x = (const E*)a.x + (long long)u * a.P * a.x_pitch + l.cv * VEC;
  const E* dy = (const E*)a.dy + (long long)u * a.P * a.dy_pitch + l.cv * VEC;
  E* dx = (E*)a.out + (long long)u * a.P * a.out_pitch + l.cv * VEC;
  Pack<T, VEC> vx[U], vd[U];
  each_row<U>(
      k * r.chunk_q + l.pl, min(r.Q, (k + 1) * r.chunk_q), r.ppi,
      [&](long long q, int i) {
        vx[i] = *(const Pack<T, VEC>*)(x + q * xp);
        vd[i] = *(const Pack<T, VEC>*)(dy + q * dp);
      },
      [&](long long q, int i) {
        float f[VEC], d[VEC];
        unpack<T, VEC>(vx[i], f);
        unpack<T, VEC>(vd[i], d);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float h, da;
          b.value(j, f[j], d[j], h, da);
          f[j] = gn_dx(b.rstd[j], b.gamma[j], da, c1[j], h, c2[j]);
        }
        store_pack<STREAM>(dx + q * op, pack<T, VEC>(f));
      });
}

// dgamma and dbeta: work-groups of 32 channels x 8 lanes of units.
__global__ __launch_bounds__(kThreads) void gn_train_params_kernel(GnTrainArgs a) {
  __shared__ double r1[8][32], r2[8][32];
  const int cl = threadIdx.x & 31, ul = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cl;
  double s1 = 0.0, s2 = 0.0;
  if (c < a.C) {
    for (int u = ul; u < a.units; u += 8) {
      s1 += a.chan[((long long)u * a.C + c) * 2];
      s2 += a.chan[((long long)u * a.C + c) * 2 + 1];
    }
  }
  r1[ul][cl] = s1;
  r2[ul][cl] = s2;
  __syncthreads();
  if (ul == 0 && c < a.C) {
    for (int i = 1; i < 8; ++i) {
      s1 += r1[i][cl];
      s2 += r2[i][cl];
    }
    if (a.dbeta) a.dbeta[c] = (float)s1;
    if (a.dgamma) a.dgamma[c] = (float)s2;
  }
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Whether every pixel row of a tensor (unit base u * P * pitch, `sp` pixels
// a row) starts at a multiple of VEC elements.
bool vector_ok(const void* p, long long pitch, int sp, int vec, int size) {
  return ((uintptr_t)p % (unsigned)(vec * size)) == 0 && (sp * pitch) % vec == 0;
}

// Rows for vectors of `vec` elements; false where the tensors do not allow
// them. A row of more than one pixel needs dense tensors, whole rows per
// unit and one channel tile.
bool rows_for(const GnTrainArgs& a, int vec, bool bwd, Rows* r) {
  const int size = elt_size(a.dtype);
  const int sp = vec / gcd(a.C, vec);
  if (sp > 1 && (a.x_pitch != a.C || (a.out && a.out_pitch != a.C) ||
                 (bwd && a.dy_pitch != a.C) || a.P % sp || sp * a.C / vec > kThreads))
    return false;
  if (!vector_ok(a.x, a.x_pitch, sp, vec, size) ||
      (a.out && !vector_ok(a.out, a.out_pitch, sp, vec, size)) ||
      (bwd && !vector_ok(a.dy, a.dy_pitch, sp, vec, size)))
    return false;
  r->sp = sp;
  r->Q = a.P / sp;
  r->chunk_q = a.chunk_px / sp;
  r->V = (int)((long long)sp * a.C / vec);
  r->tiles = (r->V + kThreads - 1) / kThreads;
  r->Vt = (r->V + r->tiles - 1) / r->tiles;
  r->ppi = kThreads / r->Vt;
  return true;
}

// Only 16-byte vectors are stored past the caches.
template <class T, int VEC>
constexpr bool kStreams = VEC * sizeof(typename T::store) == 16;

template <class T, int VEC, bool SILU>
void start_apply(const GnTrainArgs& a, const Rows& r, dim3 grid, bool stream, hipStream_t s) {
  if (stream)
    hipLaunchKernelGGL((gn_train_apply_kernel<T, VEC, SILU, kStreams<T, VEC>>), grid,
                       dim3(kThreads), 0, s, a, r);
  else
    hipLaunchKernelGGL((gn_train_apply_kernel<T, VEC, SILU, false>), grid, dim3(kThreads), 0, s, a,
                       r);
}

template <class T, int VEC>
int run_fwd(const GnTrainArgs& a, const Rows& r, hipStream_t s) {
  const dim3 grid((unsigned)a.units * (unsigned)a.chunks, r.tiles);
  hipLaunchKernelGGL((gn_train_stats_kernel<T, VEC>), grid, dim3(kThreads), 0, s, a, r);
  hipLaunchKernelGGL((gn_train_stats_finalize_kernel<T>), dim3((unsigned)a.units * (unsigned)a.G),
                     dim3(kThreads), 0, s, a);
  const bool stream = a.stream && kStreams<T, VEC>;
  if (a.silu) start_apply<T, VEC, true>(a, r, grid, stream, s);
  else start_apply<T, VEC, false>(a, r, grid, stream, s);
  return (int)hipGetLastError();
}

template <class T, int VEC, bool SILU>
int run_bwd_act(const GnTrainArgs& a, const Rows& r, hipStream_t s) {
  const dim3 grid((unsigned)a.units * (unsigned)a.chunks, r.tiles);
  hipLaunchKernelGGL((gn_train_bwd_sums_kernel<T, VEC, SILU>), grid, dim3(kThreads), 0, s, a, r);
  hipLaunchKernelGGL(gn_train_bwd_finalize_kernel, dim3((unsigned)a.units * (unsigned)a.G),
                     dim3(kThreads), 0, s, a);
  if (a.out && a.stream && kStreams<T, VEC>)
    hipLaunchKernelGGL((gn_train_bwd_apply_kernel<T, VEC, SILU, kStreams<T, VEC>>), grid,
                       dim3(kThreads), 0, s, a, r);
  else if (a.out)
    hipLaunchKernelGGL((gn_train_bwd_apply_kernel<T, VEC, SILU, false>), grid, dim3(kThreads), 0,
                       s, a, r);
  if (a.dgamma || a.dbeta)
    hipLaunchKernelGGL(gn_train_params_kernel, dim3((a.C + 31) / 32), dim3(kThreads), 0, s, a);
  return (int)hipGetLastError();
}

template <class T, int VEC>
int run_bwd(const GnTrainArgs& a, const Rows& r, hipStream_t s) {
  return a.silu ? run_bwd_act<T, VEC, true>(a, r, s) : run_bwd_act<T, VEC, false>(a, r, s);
}

// The widest of 16-byte vectors, pairs and single elements that the tensors
// allow.
template <class T>
int run(const GnTrainArgs& a, bool bwd, hipStream_t s) {
  constexpr int wide = 16 / sizeof(typename T::store);
  Rows r;
  if (rows_for(a, wide, bwd, &r))
    return bwd ? run_bwd<T, wide>(a, r, s) : run_fwd<T, wide>(a, r, s);
  if (rows_for(a, 2, bwd, &r)) return bwd ? run_bwd<T, 2>(a, r, s) : run_fwd<T, 2>(a, r, s);
  rows_for(a, 1, bwd, &r);
  return bwd ? run_bwd<T, 1>(a, r, s) : run_fwd<T, 1>(a, r, s);
}

int run_type(const GnTrainArgs& a, bool bwd, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();   // an error that another call left is not this one's
  switch (a.dtype) {
    case ELT_BF16: return run<Bf16>(a, bwd, s);
    case ELT_FP16: return run<Fp16>(a, bwd, s);
    default: return run<Fp32>(a, bwd, s);
  }
}

}  // namespace

int launch_gn_train_fwd(const GnTrainArgs& args, void* stream) {
  return run_type(args, false, stream);
}

int launch_gn_train_bwd(const GnTrainArgs& args, void* stream) {
  return run_type(args, true, stream);
}

}  // namespace conv3d
