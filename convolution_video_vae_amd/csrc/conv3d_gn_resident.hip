// Training GroupNorm (formulas in conv3d_gn_train.hip) that reads its
// activations once.
//
// A work-group keeps a piece of a unit in registers: some
// pixels of some whole groups' channels (a range). It forms the piece's
// sums, and once the sums of the whole unit are known it computes the result
// from the registers. Where a range's pixels fit one work-group (W = 1) no
// other work-group is involved. Otherwise the W pieces of a (unit, range)
// exchange their sums while all of them are on the chip: HBM then carries
// x + y instead of 2 x + y, and x + dy + dx instead of 2 x + 2 dy + dx.
//
// The exchange. Each piece publishes one 64-bit word per group (two fp32
// sums) with a relaxed agent-scope atomic store, and reads the others' words
// with relaxed atomic loads until none is the empty pattern that a kernel
// wrote before this one. A word is its own flag, so nothing has to be ordered
// against it and no cache is written back (a release per work-group would
// write back its XCD's L2).
//
// Every wait ends. A work-group polls each word at most `spin` times; if a
// word is still empty then (the other pieces cannot be resident at the same
// time: a stream confined to few CUs, other kernels that hold the chip), it
// loads the unit's other pieces itself, forms their sums with the same code
// and in the same order, and goes on. Results are therefore the same, bit
// for bit, whichever way a work-group got its sums.
#include <hip/hip_runtime.h>

#include "conv3d_colsum.h"
#include "conv3d_device.h"
#include "conv3d_elt.h"
#include "conv3d_gn_device.h"
#include "conv3d_train.h"

namespace conv3d {
namespace {

constexpr unsigned long long kEmpty = ~0ull;

// Two sums as one word that is never kEmpty: NaNs get one pattern.
__device__ __forceinline__ unsigned long long word_of(float a, float b) {
  const unsigned ua = a != a ? 0x7fc00000u : __builtin_bit_cast(unsigned, a);
  const unsigned ub = b != b ? 0x7fc00000u : __builtin_bit_cast(unsigned, b);
  return ((unsigned long long)ub << 32) | ua;
}
__device__ __forceinline__ float word_lo(unsigned long long w) {
  return __builtin_bit_cast(float, (unsigned)w);
}
__device__ __forceinline__ float word_hi(unsigned long long w) {
  return __builtin_bit_cast(float, (unsigned)(w >> 32));
}

__global__ __launch_bounds__(256) void gn_words_clear_kernel(unsigned long long* words, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) words[i] = kEmpty;
}

// A product that is never fused with a sum: pieces summed from registers and
// from memory agree bit for bit, and gamma da here is the gamma da of gn_dx.
__device__ __forceinline__ float mul_alone(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

// What a thread of a work-group holds: rows first + i * ppi, i < n, of vector
// cv of the range.
struct Where {
  int u, range, w;
  int cv, pl;
  bool active;
};

__device__ __forceinline__ Where where(const GnResPlan& r) {
  Where h;
  h.w = blockIdx.x % r.W;
  const int q = blockIdx.x / r.W;
  h.range = q % r.NR;
  h.u = q / r.NR;
  h.pl = threadIdx.x / r.Vb;
  h.cv = threadIdx.x - h.pl * r.Vb;
  h.active = h.pl < r.ppi;
  return h;
}

// The thread's rows of piece w: the first one, and how many.
__device__ __forceinline__ int rows_of(const GnTrainArgs& a, const GnResPlan& r, const Where& h,
                                       int w, long long* first) {
  const long long p0 = (long long)w * r.piece_px, p1 = min(a.P, p0 + r.piece_px);
  *first = p0 + h.pl;
  return h.active && *first < p1 ? (int)((p1 - *first + r.ppi - 1) / r.ppi) : 0;
}

template <class T, int R>
__device__ __forceinline__ void load_rows(const void* base, long long pitch, long long at,
                                          int channel0, long long first, int ppi, int n,
                                          Held<T> (&v)[R]) {
  const typename T::store* p = (const typename T::store*)base + (at + first) * pitch + channel0;
  const long long step = ppi * pitch;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < n) v[i].v = *(const u32x4_t*)p;
    p += step;
  }
}

// f(row) for the thread's n rows: the held ones, or (a work-group that helps
// itself) those of another piece, read from memory one at a time.
template <class T, int R, class F>
__device__ __forceinline__ void held_rows(const Held<T> (&v)[R], int n, F f) {
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (i < n) f(v[i]);
}
template <class T, class F>
__device__ __forceinline__ void memory_rows(const typename T::store* p, long long step, int n, F f) {
#pragma unroll 1
  for (int i = 0; i < n; ++i, p += step) {
    Held<T> v;
    v.v = *(const u32x4_t*)p;
    f(v);
  }
}

// Channel sums of N quantities over the work-group's rows: s[k][j] of every
// thread -> tot[k][channel of the range]. Rows are joined in a fixed order.
template <int NT, int N, int VEC>
struct ChannelSums {
  float red[N][NT * VEC];
  float red2[N][NT];
  float tot[N][NT];
  __device__ __forceinline__ void join(const GnResPlan& r, bool active, const float (&s)[N][VEC]) {
    const int t = threadIdx.x;
    __syncthreads();                       // the last user of these arrays is done
    if (active) {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) red[k][t * VEC + j] = s[k][j];
    }
    __syncthreads();
    const int part = t / r.Cb, col = t - part * r.Cb;
    if (part < r.parts) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        float v = 0.0f;
        for (int row = part; row < r.ppi; row += r.parts) v += red[k][row * r.Cb + col];
        red2[k][t] = v;
      }
    }
    __syncthreads();
    if (t < r.Cb) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        float v = red2[k][t];
        for (int i = 1; i < r.parts; ++i) v += red2[k][i * r.Cb + t];
        tot[k][t] = v;
      }
    }
    __syncthreads();
  }
};

// f(g, sum over group g of v(channel)) for every group of the range: by one
// thread for few channels, by a wave for many.
template <int NT, class Value, class Use>
__device__ __forceinline__ void each_group(int Gb, int cpg, Value value, Use use) {
  if (cpg <= 16) {
    for (int g = threadIdx.x; g < Gb; g += NT) {
      float v = value(g * cpg);
      for (int c = 1; c < cpg; ++c) v += value(g * cpg + c);
      use(g, v);
    }
  } else {
    const int lane = threadIdx.x & 63;
    for (int g = threadIdx.x >> 6; g < Gb; g += NT / 64) {
      float v = 0.0f;
      for (int c = lane; c < cpg; c += 64) v += value(g * cpg + c);
#pragma unroll
      for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
      if (lane == 0) use(g, v);
    }
  }
}

// The words of every piece of the (unit, range) into LDS; false where one
// stayed empty.
template <int NT>
__device__ __forceinline__ bool gather(const unsigned long long* words, int n, int spin,
                                       unsigned long long* xw, int* late) {
  for (int i = threadIdx.x; i < n; i += NT) {
    unsigned long long v = kEmpty;
    for (int k = 0; k < spin; ++k) {
      v = __hip_atomic_load(words + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (v != kEmpty) break;
      __builtin_amdgcn_s_sleep(1);
    }
    xw[i] = v;
    if (v == kEmpty) *late = 1;
  }
  __syncthreads();
  return *late == 0;
}

__device__ __forceinline__ double piece_pixels(const GnTrainArgs& a, const GnResPlan& r, int w) {
  const long long p0 = (long long)w * r.piece_px;
  return (double)(min(a.P, p0 + r.piece_px) - p0);
}

template <class T, bool SILU, int R>
__global__ __launch_bounds__(kGnResThreadsFwd, 4) void gn_resident_fwd_kernel(GnTrainArgs a, GnResPlan r) {
  typedef typename T::store E;
  constexpr int VEC = 16 / sizeof(E);
  constexpr int NT = kGnResThreadsFwd;
  __shared__ ChannelSums<NT, 1, VEC> sums;
  __shared__ unsigned long long xw[kGnResWords];
  __shared__ float gmean[NT], grstd[NT];
  __shared__ int late;
  const Where h = where(r);
  const int c0 = h.range * r.Cb + h.cv * VEC, gl0 = h.cv * VEC;
  const long long at = (long long)h.u * a.P;
  long long first;
  const int n = rows_of(a, r, h, h.w, &first);
  Held<T> v[R];
  if (threadIdx.x == 0) late = 0;

  // (mean, sum of squares about it) of a piece's groups, as words; rows(f)
  // visits the thread's rows of the piece
  const auto piece = [&](int w, unsigned long long* out, auto rows) {
    const double px = piece_pixels(a, r, w) * a.cpg;
    float s[1][VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0][j] = 0.0f;
    rows([&](const Held<T>& row) {
      float f[VEC];
      row.get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[0][j] += f[j];
    });
    sums.join(r, h.active, s);
    each_group<NT>(r.Gb, a.cpg, [&](int c) { return sums.tot[0][c]; },
               [&](int g, float t) { gmean[g] = (float)((double)t / px); });
    __syncthreads();
    float m[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      m[j] = h.active ? gmean[(gl0 + j) / a.cpg] : 0.0f;
      s[0][j] = 0.0f;
    }
    rows([&](const Held<T>& row) {
      float f[VEC];
      row.get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = f[j] - m[j];
        s[0][j] = fmaf(d, d, s[0][j]);
      }
    });
    sums.join(r, h.active, s);
    each_group<NT>(r.Gb, a.cpg, [&](int c) { return sums.tot[0][c]; },
               [&](int g, float t) { out[g] = word_of(gmean[g], t); });
    __syncthreads();
  };

  load_rows<T, R>(a.x, a.x_pitch, at, c0, first, r.ppi, n, v);
  piece(h.w, xw + h.w * r.Gb, [&](auto f) { held_rows<T, R>(v, n, f); });
  if (r.W > 1) {
    unsigned long long* words =
        r.words + ((long long)h.u * r.NR + h.range) * r.W * r.Gb;
    for (int g = threadIdx.x; g < r.Gb; g += NT)
      __hip_atomic_store(words + h.w * r.Gb + g, xw[h.w * r.Gb + g], __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (!gather<NT>(words, r.W * r.Gb, r.spin, xw, &late)) {
      for (int w = 0; w < r.W; ++w) {
        long long fw;
        const int nw = rows_of(a, r, h, w, &fw);
        const E* p = (const E*)a.x + (at + fw) * a.x_pitch + c0;
        piece(w, xw + w * r.Gb,
              [&](auto f) { memory_rows<T>(p, r.ppi * a.x_pitch, nw, f); });
      }
    }
  }
  // pieces joined in fp64: a wave per group
  for (int g = threadIdx.x >> 6; g < r.Gb; g += NT / 64) {
    const int lane = threadIdx.x & 63;
    const double N = (double)a.P * a.cpg;
    double s = 0.0;
    for (int w = lane; w < r.W; w += 64)
      s += piece_pixels(a, r, w) * a.cpg * (double)word_lo(xw[w * r.Gb + g]);
    const double mean = wave_sum(s) / N;
    s = 0.0;
    for (int w = lane; w < r.W; w += 64) {
      const double d = (double)word_lo(xw[w * r.Gb + g]) - mean;
      s += (double)word_hi(xw[w * r.Gb + g]) + piece_pixels(a, r, w) * a.cpg * d * d;
    }
    const double var = wave_sum(s) / N;
    if (lane == 0) {
      gmean[g] = (float)mean;
      grstd[g] = (float)(1.0 / sqrt(var + (double)a.eps));
    }
  }
  __syncthreads();
  if (h.w == 0) {
    float* st = a.stats + ((long long)h.u * a.G + h.range * r.Gb) * 2;
    for (int g = threadIdx.x; g < r.Gb; g += NT) {
      st[g * 2] = gmean[g];
      st[g * 2 + 1] = grstd[g];
    }
  }
  if (!h.active) return;
  float mean[VEC], scale[VEC], beta[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int g = (gl0 + j) / a.cpg;
    mean[j] = gmean[g];
    scale[j] = grstd[g] * a.gamma[c0 + j];
    beta[j] = a.beta[c0 + j];
  }
  E* y = (E*)a.out + (at + first) * a.out_pitch + c0;
  const long long step = r.ppi * a.out_pitch;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    __builtin_amdgcn_sched_barrier(0);
    if (i < n) {
      float f[VEC];
      v[i].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        f[j] = fmaf(f[j] - mean[j], scale[j], beta[j]);
        if (SILU) f[j] = silu_of<T::kWide>(f[j]);
      }
      Held<T> o;
      o.put(f);
      *(u32x4_t*)y = o.v;
    }
    y += step;
  }
}

template <class T, bool SILU, int R>
__global__ __launch_bounds__(kGnResThreadsBwd, 2) void gn_resident_bwd_kernel(GnTrainArgs a, GnResPlan r) {
  typedef typename T::store E;
  constexpr int VEC = 16 / sizeof(E);
  constexpr int NT = kGnResThreadsBwd;
  __shared__ ChannelSums<NT, 2, VEC> sums;
  __shared__ unsigned long long xw[kGnResWords];
  __shared__ float g1[NT], g2[NT];
  __shared__ int late;
  const Where h = where(r);
  const int c0 = h.range * r.Cb + h.cv * VEC, gl0 = h.cv * VEC;
  const long long at = (long long)h.u * a.P;
  const float* st = a.stats + ((long long)h.u * a.G + h.range * r.Gb) * 2;
  long long first;
  const int n = rows_of(a, r, h, h.w, &first);
  Held<T> vx[R], vd[R];
  float mean[VEC], rstd[VEC], gamma[VEC], beta[VEC];
  if (threadIdx.x == 0) late = 0;
  load_rows<T, R>(a.x, a.x_pitch, at, c0, first, r.ppi, n, vx);
  load_rows<T, R>(a.dy, a.dy_pitch, at, c0, first, r.ppi, n, vd);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int g = h.active ? (gl0 + j) / a.cpg : 0, c = h.active ? c0 + j : 0;
    mean[j] = st[g * 2];
    rstd[j] = st[g * 2 + 1];
    gamma[j] = a.gamma[c];
    beta[j] = a.beta[c];
  }
  const auto value = [&](int j, float x, float dy, float& hh, float& da) {
    hh = mul_alone(x - mean[j], rstd[j]);
    da = SILU ? mul_alone(dy, silu_slope<T::kWide>(fmaf(hh, gamma[j], beta[j]))) : dy;
  };
  // (sum of gamma da, of gamma da h) of a piece's groups, as words
  const auto piece = [&](unsigned long long* out, auto rows) {
    float s[2][VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0][j] = s[1][j] = 0.0f;
    rows([&](const Held<T>& rx, const Held<T>& rd) {
      float f[VEC], d[VEC];
      rx.get(f);
      rd.get(d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float hh, da;
        value(j, f[j], d[j], hh, da);
        s[0][j] = fmaf(da, hh, s[0][j]);
        s[1][j] += da;
      }
    });
    sums.join(r, h.active, s);
    const float* gm = a.gamma + h.range * r.Cb;
    each_group<NT>(r.Gb, a.cpg, [&](int c) { return mul_alone(gm[c], sums.tot[1][c]); },
               [&](int g, float t) { g1[g] = t; });
    each_group<NT>(r.Gb, a.cpg, [&](int c) { return mul_alone(gm[c], sums.tot[0][c]); },
               [&](int g, float t) { g2[g] = t; });
    __syncthreads();
    for (int g = threadIdx.x; g < r.Gb; g += NT) out[g] = word_of(g1[g], g2[g]);
  };
  piece(xw + h.w * r.Gb, [&](auto f) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i < n) f(vx[i], vd[i]);
  });
  if (r.channel_sums) {
    float* row = r.channel_sums + ((long long)h.u * r.W + h.w) * 2 * a.C + h.range * r.Cb;
    if (threadIdx.x < r.Cb) {
      row[threadIdx.x] = sums.tot[0][threadIdx.x];
      row[a.C + threadIdx.x] = sums.tot[1][threadIdx.x];
    }
  }
  if (!a.out) return;
  __syncthreads();
  if (r.W > 1) {
    unsigned long long* words =
        r.words + ((long long)h.u * r.NR + h.range) * r.W * r.Gb;
    for (int g = threadIdx.x; g < r.Gb; g += NT)
      __hip_atomic_store(words + h.w * r.Gb + g, xw[h.w * r.Gb + g], __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (!gather<NT>(words, r.W * r.Gb, r.spin, xw, &late)) {
      for (int w = 0; w < r.W; ++w) {
        long long fw;
        const int nw = rows_of(a, r, h, w, &fw);
        const E* px = (const E*)a.x + (at + fw) * a.x_pitch + c0;
        const E* pd = (const E*)a.dy + (at + fw) * a.dy_pitch + c0;
        piece(xw + w * r.Gb, [&](auto f) {
#pragma unroll 1
          for (int i = 0; i < nw; ++i) {
            Held<T> x1, d1;
            x1.v = *(const u32x4_t*)(px + i * (r.ppi * a.x_pitch));
            d1.v = *(const u32x4_t*)(pd + i * (r.ppi * a.dy_pitch));
            f(x1, d1);
          }
        });
      }
      __syncthreads();
    }
  }
  for (int g = threadIdx.x >> 6; g < r.Gb; g += NT / 64) {
    const int lane = threadIdx.x & 63;
    const double N = (double)a.P * a.cpg;
    double s1 = 0.0, s2 = 0.0;
    for (int w = lane; w < r.W; w += 64) {
      s1 += (double)word_lo(xw[w * r.Gb + g]);
      s2 += (double)word_hi(xw[w * r.Gb + g]);
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if (lane == 0) {
      g1[g] = (float)(s1 / N);
      g2[g] = (float)(s2 / N);
    }
  }
  __syncthreads();
  if (!h.active) return;
  float c1[VEC], c2[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    c1[j] = g1[(gl0 + j) / a.cpg];
    c2[j] = g2[(gl0 + j) / a.cpg];
  }
  E* dx = (E*)a.out + (at + first) * a.out_pitch + c0;
  const long long step = r.ppi * a.out_pitch;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    __builtin_amdgcn_sched_barrier(0);
    if (i < n) {
      float f[VEC], d[VEC];
      vx[i].get(f);
      vd[i].get(d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float hh, da;
        value(j, f[j], d[j], hh, da);
        f[j] = gn_dx(rstd[j], gamma[j], da, c1[j], hh, c2[j]);
      }
      Held<T> o;
      o.put(f);
      *(u32x4_t*)dx = o.v;
    }
    dx += step;
  }
}

void clear_words(const GnTrainArgs& a, const GnResPlan& r, hipStream_t s) {
  const int n = a.units * r.NR * r.W * r.Gb;
  hipLaunchKernelGGL(gn_words_clear_kernel, dim3((n + 255) / 256), dim3(256), 0, s, r.words, n);
}

template <class T, bool SILU>
int run_fwd(const GnTrainArgs& a, const GnResPlan& r, hipStream_t s) {
  if (r.W > 1) clear_words(a, r, s);
  const dim3 grid(a.units * r.NR * r.W);
  const dim3 block(kGnResThreadsFwd);
  if (r.passes <= 4)
    hipLaunchKernelGGL((gn_resident_fwd_kernel<T, SILU, 4>), grid, block, 0, s, a, r);
  else
    hipLaunchKernelGGL((gn_resident_fwd_kernel<T, SILU, kGnResRows>), grid, block, 0, s, a, r);
  return (int)hipGetLastError();
}

template <class T, bool SILU>
int run_bwd(const GnTrainArgs& a, const GnResPlan& r, hipStream_t s) {
  if (r.W > 1 && a.out) clear_words(a, r, s);
  const dim3 grid(a.units * r.NR * r.W);
  const dim3 block(kGnResThreadsBwd);
  if (r.passes <= 4)
    hipLaunchKernelGGL((gn_resident_bwd_kernel<T, SILU, 4>), grid, block, 0, s, a, r);
  else
    hipLaunchKernelGGL((gn_resident_bwd_kernel<T, SILU, kGnResRows>), grid, block, 0, s, a, r);
  if (r.channel_sums)
    hipLaunchKernelGGL(column_sums_kernel, dim3((2 * a.C + kSumCols - 1) / kSumCols),
                       dim3(kSumThreads), 0, s, r.channel_sums, a.units * r.W, a.C, a.dgamma,
                       a.dbeta);
  return (int)hipGetLastError();
}

template <class T>
int run(const GnTrainArgs& a, const GnResPlan& r, bool bwd, hipStream_t s) {
  if (bwd) return a.silu ? run_bwd<T, true>(a, r, s) : run_bwd<T, false>(a, r, s);
  return a.silu ? run_fwd<T, true>(a, r, s) : run_fwd<T, false>(a, r, s);
}

}  // namespace

int launch_gn_resident(const GnTrainArgs& a, const GnResPlan& r, bool bwd, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  switch (a.dtype) {
    case ELT_BF16: return run<Bf16>(a, r, bwd, s);
    case ELT_FP16: return run<Fp16>(a, r, bwd, s);
    default: return run<Fp32>(a, r, bwd, s);
  }
}

}  // namespace conv3d
