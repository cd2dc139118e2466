// Training GroupNorm (formulas in conv3d_gn_train.hip) that reads its
// activations once.
//
// A work-group keeps a piece of a unit in registers and LDS: some pixels of
// some whole groups' channels (a range). It forms the piece's sums, and once
// the sums of the whole unit are known it computes the result from what it
// holds. Where a range's pixels fit one work-group (W = 1) no
// other work-group is involved. Otherwise the W pieces of a (unit, range)
// exchange their sums while all of them are on the chip: HBM then carries
// x + y instead of 2 x + y, and x + dy + dx instead of 2 x + 2 dy + dx.
//
// Rows are loaded as non-temporal: they are read once, and what they would
// push out of the memory-side cache are dirty lines of y or dx, whose
// write-back then competes with the loads (H3 L0 forward 134 -> 128 us,
// backward 218 -> 209 us when this came in). So are results stored that would
// fill half of that cache and more (128 -> 121 and 209 -> 205 us); smaller ones
// stay there for their reader. H3 L0 now: 121 and 196 us, 91 and 85 % of a
// copy's rate.
//
// The exchange. Each piece publishes one 64-bit word per group (two fp32
// sums) with a relaxed agent-scope atomic store, and reads the others' words
// with relaxed atomic loads until none is the empty pattern that a kernel
// wrote before this one. A word is its own flag, so nothing has to be ordered
// against it and no cache is written back (a release per work-group would
// write back its XCD's L2).
//
// Every wait ends. A thread polls at most `spin` times for all its words
// together; if one is still empty then (the other pieces cannot be resident at the same
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

typedef float f32x2_t __attribute__((ext_vector_type(2)));

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

// STREAM is a template argument: the compiler joins the two stores of a branch
// into an ordinary one.
template <bool STREAM>
__device__ __forceinline__ void store_row(void* p, const u32x4_t& v) {
  if (STREAM) __builtin_nontemporal_store(v, (u32x4_t*)p);
  else *(u32x4_t*)p = v;
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

// Group of element j of a thread's vector whose first channel (of the range)
// is c: one division, then counting.
struct GroupOf {
  int g, left;
  __device__ __forceinline__ GroupOf(int c, int cpg) : g(c / cpg), left(cpg - (c - c / cpg * cpg)) {}
  __device__ __forceinline__ int next(int cpg) {
    const int now = g;
    if (--left == 0) {
      ++g;
      left = cpg;
    }
    return now;
  }
};

// ---- joining a work-group's rows
//
// Where a row's vectors are a power of two of lanes, rows of one wave are
// joined by exchanges between lanes and only one value per wave goes through
// LDS; else every lane's goes. Either way in a fixed order. Rows of at most 16
// lanes leave a quarter of the values to each quarter of the wave: 16 values of
// 8 lanes take 16 exchanges instead of 48. (With da and h kept where R <= 4 and
// both sums of a group in one pass: H3 L0 backward 205 -> 194.5 us,
// [1,5,16,16,1024] bf16 backward 12.1 -> 9.3 us.)

// Lanes below 32: the sum of a of lane and lane + 32; the others: of b of lane
// and lane - 32. (The elements are copied first: a bit cast of one in place
// reads element 0.)
__device__ __forceinline__ float halves(float a, float b) {
  const auto v = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, a),
                                                  __builtin_bit_cast(unsigned, b), false, false);
  const unsigned lo = v[0], hi = v[1];
  return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}
// The same between the two rows of 16 lanes of each half.
__device__ __forceinline__ float rows16(float a, float b) {
  const auto v = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a),
                                                  __builtin_bit_cast(unsigned, b), false, false);
  const unsigned lo = v[0], hi = v[1];
  return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}

// Channel sums of two quantities: s[k][j] of every thread -> tot(channel, v0, v1)
// by the thread of that number.
// COMPACT (the lanes' form, at most kGnCompact values of a row): small arrays,
// and the space is left to rows.
template <int NT, int VEC, bool COMPACT>
struct ChannelSums {
  float red[2][COMPACT ? NT / 64 * kGnCompact : NT * VEC];
  template <class Tot>
  __device__ __forceinline__ void join(const GnResPlan& r, bool active, float (&s)[2][VEC],
                                       Tot tot) {
    const int t = threadIdx.x;
    const bool lanes = COMPACT || r.lanes;
    const bool quarters = lanes && r.Vb <= 16;
    if (quarters) {
      // two quantities' halves of the wave change places and are added: a
      // quarter of the wave is left with a quarter of the values
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[0][j] = halves(s[0][j], s[1][j]);
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) s[0][j] = rows16(s[0][j], s[0][j + VEC / 2]);
      for (int m = r.Vb; m < 16; m <<= 1)
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) s[0][j] += __shfl_xor(s[0][j], m);
    } else if (lanes) {
      for (int m = r.Vb; m < 64; m <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < VEC; ++j) s[k][j] += __shfl_xor(s[k][j], m);
    }
    const int rows = lanes ? NT / 64 : r.ppi;
    const int at = lanes ? (t >> 6) * r.Cb + (t & (quarters ? 15 : 63)) * VEC : t * VEC;
    if (quarters) {
      if ((t & 15) < r.Vb)
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j)
          red[(t >> 5) & 1][at + (t & 16 ? VEC / 2 : 0) + j] = s[0][j];
    } else if (lanes ? (t & 63) < r.Vb : active) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) red[k][at + j] = s[k][j];
    }
    __syncthreads();
    if (t < r.Cb) {
      float v0 = red[0][t], v1 = red[1][t];
      for (int i = 1; i < rows; ++i) {
        v0 += red[0][i * r.Cb + t];
        v1 += red[1][i * r.Cb + t];
      }
      tot(t, v0, v1);
    }
  }
};

// A sample of n values: their mean and the squares' sum about it. Two are
// joined by Chan, Golub and LeVeque's update; nothing cancels.
struct Moments {
  float mean, m2;
  __device__ __forceinline__ void join(float n, const Moments& o, float on) {
    const float total = n + on;
    const float d = o.mean - mean;
    const float share = total > 0.0f ? on * __builtin_amdgcn_rcpf(total) : 0.0f;
    m2 = m2 + o.m2 + d * d * (n * share);
    mean = fmaf(d, share, mean);
  }
};

// (mean, squares about it) of the groups of a piece to use(g, mean, m2), from
// one Moments per slot (`fold` channels of one group) and wave (or lane row).
template <int NT, int VEC, bool COMPACT>
struct GroupMoments {
  static constexpr int kSize = COMPACT ? NT / 64 * kGnCompact : NT * VEC;
  float mean[kSize], m2[kSize];
  float n[NT];
  template <class Use>
  __device__ __forceinline__ void join(const GnResPlan& r, int cpg, bool active, int rows,
                                       Moments (&s)[VEC], Use use) {
    const int t = threadIdx.x;
    float cnt = (float)rows;
    // channels of one group in the vector: equal counts
#pragma unroll
    for (int f = 1; f < VEC; f *= 2)
      if (r.fold > f) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2 * f) {
          const float d = s[j + f].mean - s[j].mean;
          s[j].m2 = s[j].m2 + s[j + f].m2 + d * d * (0.5f * cnt);
          s[j].mean = fmaf(0.5f, d, s[j].mean);
        }
        cnt *= 2.0f;
      }
    const bool lanes = COMPACT || r.lanes;
    if (lanes) {
      for (int m = r.Vb; m < 64; m <<= 1) {
        const float on = __shfl_xor(cnt, m);
        const bool low = (t & m) == 0;          // both lanes join in the same order
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          if (j & (r.fold - 1)) continue;
          Moments o;
          o.mean = __shfl_xor(s[j].mean, m);
          o.m2 = __shfl_xor(s[j].m2, m);
          Moments a = low ? s[j] : o;
          const Moments b = low ? o : s[j];
          a.join(low ? cnt : on, b, low ? on : cnt);
          s[j] = a;
        }
        cnt += on;
      }
    }
    const int nrow = lanes ? NT / 64 : r.ppi;
    const int slots = VEC / r.fold;             // of a thread's vector
    const int width = r.Vb * slots;
    const int lane = lanes ? t & 63 : t % r.Vb, row = lanes ? t >> 6 : t / r.Vb;
    if (lanes ? lane < r.Vb : active) {
      n[row * r.Vb + lane] = cnt;
      int at = row * width + lane * slots;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (j & (r.fold - 1)) continue;
        mean[at] = s[j].mean;
        m2[at] = s[j].m2;
        ++at;
      }
    }
    __syncthreads();
    // a group's entries (of its slots and the rows) over a few lanes, and those
    const int per = cpg / r.fold, lg = r.entry_lanes, sub = t & (lg - 1);
    for (int g = t / lg; g < r.Gb; g += NT / lg) {
      Moments q = {0.0f, 0.0f};
      float qn = 0.0f;
      int i = sub / per, k = sub - i * per;
      for (int e = sub; e < nrow * per; e += lg) {
        const int slot = g * per + k;
        const float on = n[i * r.Vb + slot / slots];
        q.join(qn, Moments{mean[i * width + slot], m2[i * width + slot]}, on);
        qn += on;
        for (k += lg; k >= per; k -= per) ++i;
      }
      for (int m = lg >> 1; m > 0; m >>= 1) {
        Moments o;
        o.mean = __shfl_xor(q.mean, m);
        o.m2 = __shfl_xor(q.m2, m);
        const float on = __shfl_xor(qn, m);
        const bool low = (sub & m) == 0;
        Moments a = low ? q : o;
        a.join(low ? qn : on, low ? o : q, low ? on : qn);
        q = a;
        qn += on;
      }
      if (sub == 0) use(g, q.mean, q.m2);
    }
  }
};

// use(g, the sums over group g of the two values of v(channel)) for every group
// of the range: by one thread for few channels, by a wave for many.
template <int NT, class Value, class Use>
__device__ __forceinline__ void each_group(int Gb, int cpg, Value value, Use use) {
  if (cpg <= 16) {
    for (int g = threadIdx.x; g < Gb; g += NT) {
      f32x2_t v = value(g * cpg);
      for (int c = 1; c < cpg; ++c) {
        const f32x2_t o = value(g * cpg + c);
        v[0] += o[0];
        v[1] += o[1];
      }
      use(g, v);
    }
  } else {
    const int lane = threadIdx.x & 63;
    for (int g = threadIdx.x >> 6; g < Gb; g += NT / 64) {
      f32x2_t v = {0.0f, 0.0f};
      for (int c = lane; c < cpg; c += 64) {
        const f32x2_t o = value(g * cpg + c);
        v[0] += o[0];
        v[1] += o[1];
      }
#pragma unroll
      for (int m = 32; m > 0; m >>= 1) {
        v[0] += __shfl_xor(v[0], m);
        v[1] += __shfl_xor(v[1], m);
      }
      if (lane == 0) use(g, v);
    }
  }
}

// ---- the exchange

// Sums over the pieces of a (unit, range), in fp64. Thread t takes group t %
// Gb and every LG-th piece from t / Gb on (LG = NT / Gb), so a work-group's
// reads of the words are contiguous; the threads' sums are joined in order.
template <int NT>
struct PieceSums {
  union {
    double a[NT];
    f32x4_t ref[NT / 4];         // before the join: the channels' reference values
  };
  double b[NT];
  unsigned long long own[NT];    // one piece's words
  int late;

  // Publishes this piece's words (in own, visible to all threads) and calls
  // add(w, word) for the thread's group and pieces in ascending order; false
  // where a piece's word stayed empty, and then nothing is to be believed.
  template <class Add>
  __device__ __forceinline__ bool collect(const GnResPlan& r, const Where& h, Add add) {
    const int t = threadIdx.x;
    unsigned long long* words = r.words + ((long long)h.u * r.NR + h.range) * r.W * r.Gb;
    if (t == 0) late = 0;
    for (int g = t; g < r.Gb; g += NT)
      __hip_atomic_store(words + h.w * r.Gb + g, own[g], __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const int LG = NT / r.Gb, slot = t / r.Gb, g = t - slot * r.Gb;
    // two words in flight per thread: a poll is a trip to memory, behind the
    // rows that the other work-group on this CU has asked for
    int left = r.spin;
    for (int w0 = slot < LG ? slot : r.W; w0 < r.W; w0 += 2 * LG) {
      const int w1 = w0 + LG;
      bool open0 = w0 != h.w, open1 = w1 < r.W && w1 != h.w;
      unsigned long long v0 = own[g], v1 = v0;
      for (; left > 0 && (open0 | open1); --left) {
        if (open0)
          v0 = __hip_atomic_load(words + w0 * r.Gb + g, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (open1)
          v1 = __hip_atomic_load(words + w1 * r.Gb + g, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        open0 = open0 && v0 == kEmpty;
        open1 = open1 && v1 == kEmpty;
      }
      if (open0 | open1) late = 1;
      add(w0, v0);
      if (w1 < r.W) add(w1, v1);
    }
    __syncthreads();
    return late == 0;
  }

  // add() of one piece whose words have been left in own, for the threads that
  // take it.
  template <class Add>
  __device__ __forceinline__ void one(const GnResPlan& r, int w, Add add) {
    __syncthreads();
    const int LG = NT / r.Gb, slot = threadIdx.x / r.Gb;
    if (slot < LG && w % LG == slot) add(w, own[threadIdx.x - slot * r.Gb]);
    __syncthreads();
  }

  // The threads' sums joined per group, to use(g, sum, sum).
  template <class Use>
  __device__ __forceinline__ void join(const GnResPlan& r, double s1, double s2, Use use) {
    const int t = threadIdx.x;
    a[t] = s1;
    b[t] = s2;
    __syncthreads();
    const int LG = min(NT / r.Gb, r.W);
    if (LG <= 32) {
      for (int g = t; g < r.Gb; g += NT) {
        double x = a[g], y = b[g];
        for (int i = 1; i < LG; ++i) {
          x += a[i * r.Gb + g];
          y += b[i * r.Gb + g];
        }
        use(g, x, y);
      }
    } else {
      for (int g = t >> 6; g < r.Gb; g += NT / 64) {
        double x = 0.0, y = 0.0;
        for (int i = t & 63; i < LG; i += 64) {
          x += a[i * r.Gb + g];
          y += b[i * r.Gb + g];
        }
        x = wave_sum(x);
        y = wave_sum(y);
        if ((t & 63) == 0) use(g, x, y);
      }
    }
    __syncthreads();
  }
};

// Steps of a vector's values are kept apart from each other: the compiler
// would chain one value's exponential and reciprocal after another's to save
// registers, and wait for each (two waves per SIMD hide nothing: 7.5 us of a
// piece's 23).
__device__ __forceinline__ void step_edge() { __builtin_amdgcn_sched_barrier(0); }

// R rows of which LROWS are kept in LDS.
template <class T, bool SILU, int R, int LROWS, bool COMPACT, bool STREAM>
__global__ __launch_bounds__(kGnResThreadsFwd, 4) void gn_resident_fwd_kernel(GnTrainArgs a,
                                                                              GnResPlan r) {
  typedef typename T::store E;
  constexpr int VEC = 16 / sizeof(E), NT = kGnResThreadsFwd;
  __shared__ GroupMoments<NT, VEC, COMPACT> sums;
  __shared__ u32x4_t lds_x[LROWS ? LROWS : 1][LROWS ? NT : 1];
  __shared__ PieceSums<NT> pieces;
  __shared__ float gmean[NT], grstd[NT];
  __shared__ float lgamma[NT], lbeta[NT];
  const Where h = where(r);
  // ahead of the rows: a load that is issued later returns after all of them,
  // and after those of the other work-group on this CU
  const int ct = min((int)threadIdx.x, r.Cb - 1), kg = ct / a.cpg;
  const float gamma_t = a.gamma[h.range * r.Cb + ct], beta_t = a.beta[h.range * r.Cb + ct];
  const int c0 = h.range * r.Cb + h.cv * VEC, gl0 = h.cv * VEC;
  const long long at = (long long)h.u * a.P;
  Samples<T> near;
  near.load((const E*)a.x + at * a.x_pitch + h.range * r.Cb + kg * a.cpg, a.P, a.x_pitch, a.cpg);
  long long first;
  const int n = rows_of(a, r, h, h.w, &first);
  Held<T> v[R];

  // Per channel, sums about the thread's first value (no cancellation where
  // the mean is far above the spread) -> the piece's group moments as words,
  // the mean from the group's reference value on (in gmean too, until the mean
  // is known): joined as they are, means far above the spread would take a
  // rounding of their own size at every join.
  // rows(f) visits the thread's rows of the piece, use(g, word) takes the words.
  const auto piece = [&](int n, const Held<T>& v0, auto rows, auto use) {
    float sh[VEC], s1[VEC], s2[VEC];
    v0.get(sh);
#pragma unroll
    for (int j = 0; j < VEC; ++j) s1[j] = s2[j] = 0.0f;
    rows([&](const Held<T>& row) {
      float f[VEC];
      row.get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = f[j] - sh[j];
        s1[j] += d;
        s2[j] = fmaf(d, d, s2[j]);
      }
    });
    Moments m[VEC];
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
    f32x4_t ref[VEC / 4];
#pragma unroll
    for (int j = 0; j < VEC; j += 4) ref[j / 4] = pieces.ref[(gl0 + j) / 4];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float d = s1[j] * inv, mean = (sh[j] - ref[j / 4][j & 3]) + d;
      m[j].mean = n > 0 ? mean : 0.0f;
      m[j].m2 = fmaf(-d, s1[j], s2[j]);
      m[j].m2 = m[j].m2 < 0.0f ? 0.0f : m[j].m2;      // and not fmaxf: a NaN stays
    }
    sums.join(r, a.cpg, h.active, n, m, [&](int g, float mu, float q) { use(g, word_of(mu, q)); });
  };

  {
    const E* p = (const E*)a.x + (at + first) * a.x_pitch + c0;
    const long long step = r.ppi * a.x_pitch;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      v[i].v = u32x4_t{0, 0, 0, 0};
      if (i < n) v[i].v = __builtin_nontemporal_load((const u32x4_t*)p);
      p += step;
    }
  }
  if (threadIdx.x < r.Cb) {
    const float k = near.reference();
    lgamma[threadIdx.x] = gamma_t;
    lbeta[threadIdx.x] = beta_t;
    ((float*)pieces.ref)[threadIdx.x] = k;
    if (threadIdx.x == kg * a.cpg) gmean[kg] = k;
  }
  // pieces joined by the sums of n mean and of squares + n mean^2 (the counts
  // are formed where they are used: six registers less beside the rows)
  const auto values = [&](int w) {
    return (double)(w == r.W - 1 ? a.P - (long long)w * r.piece_px : r.piece_px) * a.cpg;
  };
  const auto group = [&](int g, double s1, double s2) {
    const double inv_n = 1.0 / ((double)a.P * a.cpg);
    const double mean = s1 * inv_n, var = s2 * inv_n - mean * mean;
    gmean[g] = (float)((double)gmean[g] + mean);
    grstd[g] = (float)(1.0 / sqrt((var < 0.0 ? 0.0 : var) + (double)a.eps));  // a NaN stays
  };
  piece(
      n, v[0],
      [&](auto f) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          if (i < n) f(v[i]);
          if (i < LROWS) lds_x[i][threadIdx.x] = v[i].v;
        }
        __syncthreads();   // pieces.ref
      },
      [&](int g, unsigned long long word) {
        if (r.W > 1) {
          pieces.own[g] = word;
        } else {
          const double mean = word_lo(word), N = values(0);
          group(g, mean * N, (double)word_hi(word) + mean * mean * N);
        }
      });
  __syncthreads();
  if (r.W > 1) {
    double s1 = 0.0, s2 = 0.0;
    const auto add = [&](int w, unsigned long long x) {
      const double mean = word_lo(x), nm = values(w) * mean;
      s1 += nm;
      s2 += (double)word_hi(x) + nm * mean;
    };
    if (!pieces.collect(r, h, add)) {
      s1 = s2 = 0.0;
      for (int w = 0; w < r.W; ++w) {
        long long fw;
        const int nw = rows_of(a, r, h, w, &fw);
        const E* p = (const E*)a.x + (at + fw) * a.x_pitch + c0;
        const long long step = r.ppi * a.x_pitch;
        Held<T> v0;
        v0.v = u32x4_t{0, 0, 0, 0};
        if (nw > 0) v0.v = *(const u32x4_t*)p;
        piece(
            nw, v0,
            [&](auto f) {
#pragma unroll 1
              for (int i = 0; i < nw; ++i) {
                Held<T> row;
                row.v = *(const u32x4_t*)(p + i * step);
                f(row);
              }
            },
            [&](int g, unsigned long long word) { pieces.own[g] = word; });
        pieces.one(r, w, add);
      }
    }
    pieces.join(r, s1, s2, group);
  }
  if (h.w == 0) {
    float* st = a.stats + ((long long)h.u * a.G + h.range * r.Gb) * 2;
    for (int g = threadIdx.x; g < r.Gb; g += NT) {
      st[g * 2] = gmean[g];
      st[g * 2 + 1] = grstd[g];
    }
  }
  if (!h.active) return;
  // The difference from the mean first: x scale + (beta - mean scale) in one
  // product would leave a rounding of mean scale, and scale is 316 gamma in a
  // constant group. (A product costs [1,9,128,128,320] fp16 61.9 instead of 63 us,
  // H3 L0 nothing.)
  float mean[VEC], scale[VEC], beta[VEC];
  GroupOf go(gl0, a.cpg);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int g = go.next(a.cpg);
    mean[j] = gmean[g];
    scale[j] = grstd[g] * lgamma[gl0 + j];
    beta[j] = lbeta[gl0 + j];
  }
  // the thread's place once more: kept since the loads, it spills
  int t = threadIdx.x;
  asm("" : "+v"(t));
  const int pl = t / r.Vb;
  E* y = (E*)a.out + (at + (long long)h.w * r.piece_px + pl) * a.out_pitch + h.range * r.Cb +
         (t - pl * r.Vb) * VEC;
  const long long step = r.ppi * a.out_pitch;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < n) {
      float f[VEC];
      if (i < LROWS) v[i].v = lds_x[i][threadIdx.x];
      v[i].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        f[j] = fmaf(f[j] - mean[j], scale[j], beta[j]);
        if (SILU && T::kWide) f[j] = silu_of<true>(f[j]);
      }
      if (SILU && !T::kWide) {
        constexpr float kLog2e = 1.44269502162933349609375f;
        float t[VEC];
        step_edge();
#pragma unroll
        for (int j = 0; j < VEC; ++j) t[j] = __builtin_amdgcn_exp2f(-f[j] * kLog2e);
        step_edge();
#pragma unroll
        for (int j = 0; j < VEC; ++j) t[j] = __builtin_amdgcn_rcpf(1.0f + t[j]);
        step_edge();
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] *= t[j];
      }
      Held<T> o;
      o.put(f);
      store_row<STREAM>(y, o.v);
    }
    y += step;
  }
}

// h and da of a vector from its channels' constants. 16-bit types: a sigmoid's
// argument straight in powers of two (p = -a log2 e), and 1 + a (1 - sigmoid)
// from p. fp32: as the formulas say. The difference from the mean always comes
// first: x rstd - mean rstd in one product would leave a rounding of mean rstd,
// and in a constant group, where h is 0, nothing else. (That product took 95 us
// instead of 98.5 on [1,17,128,128,256] fp16, 193 instead of 196 on
// [1,17,256,256,128] bf16.)
template <class T, bool SILU, int VEC, int GV>
struct BwdValues {
  float mean[GV], rstd[GV], gamma[VEC], beta[VEC];
  static constexpr int at(int j) { return j * GV / VEC; }
  __device__ __forceinline__ void init(int j, float m, float s, float g, float b) {
    constexpr float kLog2e = 1.44269502162933349609375f;
    mean[at(j)] = m;
    rstd[at(j)] = s;
    gamma[j] = T::kWide ? g : -g * kLog2e;
    beta[j] = T::kWide ? b : -b * kLog2e;
  }
  __device__ __forceinline__ float h(int j, float x) const {
    return mul_alone(x - mean[at(j)], rstd[at(j)]);
  }
  // x becomes h, dy becomes da
  __device__ __forceinline__ void run(float (&x)[VEC], float (&dy)[VEC]) const {
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = h(j, x[j]);
    if (!SILU) return;
    if (T::kWide) {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        dy[j] = mul_alone(dy[j], silu_slope<true>(fmaf(x[j], gamma[j], beta[j])));
      return;
    }
    constexpr float kLn2 = 0.693147182464599609375f;
    float p[VEC], t[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) p[j] = fmaf(x[j], gamma[j], beta[j]);
    step_edge();
#pragma unroll
    for (int j = 0; j < VEC; ++j) t[j] = __builtin_amdgcn_exp2f(p[j]);
    step_edge();
#pragma unroll
    for (int j = 0; j < VEC; ++j) t[j] += 1.0f;
    step_edge();
#pragma unroll
    for (int j = 0; j < VEC; ++j) t[j] = __builtin_amdgcn_rcpf(t[j]);
    step_edge();
#pragma unroll
    for (int j = 0; j < VEC; ++j) p[j] = fmaf(p[j], fmaf(t[j], kLn2, -kLn2), 1.0f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) dy[j] = mul_alone(dy[j], t[j] * p[j]);
    step_edge();
  }
};

// R <= 4 rows: few values, where the terms of dx may cancel: gn_dx, of da and h
// as they were. More rows: da is kept in the place of dy, of LROWS rows in LDS,
// and dx is two products per value. GV groups at most share a vector's channels: VEC, or
// a quarter of that where every four channels are of one group.
template <class T, bool SILU, int R, int LROWS, int GV, bool COMPACT, bool STREAM>
__global__ __launch_bounds__(kGnResThreadsBwd, 2) void gn_resident_bwd_kernel(GnTrainArgs a,
                                                                              GnResPlan r) {
  typedef typename T::store E;
  constexpr int VEC = 16 / sizeof(E), NT = kGnResThreadsBwd;
  constexpr bool FEW = R <= 4;
  __shared__ ChannelSums<NT, VEC, COMPACT> sums;
  __shared__ float tot[2][NT];
  __shared__ PieceSums<NT> pieces;
  __shared__ f32x4_t lds_da[LROWS ? LROWS : 1][VEC / 4][LROWS ? NT : 1];
  __shared__ float g1[NT], g2[NT], lgamma[NT];
  const Where h = where(r);
  const int c0 = h.range * r.Cb + h.cv * VEC, gl0 = h.cv * VEC;
  const long long at = (long long)h.u * a.P;
  const float* st = a.stats + ((long long)h.u * a.G + h.range * r.Gb) * 2;
  long long first;
  const int n = rows_of(a, r, h, h.w, &first);
  Held<T> vx[R], vd[R];
  float vda[R - LROWS][VEC], vh[FEW ? R : 1][VEC];
  BwdValues<T, SILU, VEC, GV> bv;
  // ahead of the rows, as in the forward pass
  if (threadIdx.x < r.Cb) lgamma[threadIdx.x] = a.gamma[h.range * r.Cb + threadIdx.x];
  {
    GroupOf go(h.active ? gl0 : 0, a.cpg);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int g = go.next(a.cpg), c = h.active ? c0 + j : 0;
      bv.init(j, st[g * 2], st[g * 2 + 1], a.gamma[c], a.beta[c]);
    }
  }
  {
    const E* px = (const E*)a.x + (at + first) * a.x_pitch + c0;
    const E* pd = (const E*)a.dy + (at + first) * a.dy_pitch + c0;
    const long long sx = r.ppi * a.x_pitch, sd = r.ppi * a.dy_pitch;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i < n) {
        vx[i].v = __builtin_nontemporal_load((const u32x4_t*)px);
        vd[i].v = __builtin_nontemporal_load((const u32x4_t*)pd);
      }
      px += sx;
      pd += sd;
    }
  }
  // (sum of gamma da, of gamma da h) of a piece's groups, as words to use(g,
  // word): where a group is a power of two of a wave's lanes, from its channels'
  // threads without another barrier ([8,5,32,32,512] bf16 39.6 -> 38.6 us)
  const bool within = a.cpg <= 64 && (a.cpg & (a.cpg - 1)) == 0;
  const auto piece = [&](float (&s)[2][VEC], auto channel, auto use) {
    sums.join(r, h.active, s, [&](int c, float dah, float da) {
      channel(c, dah, da);
      float w1 = mul_alone(lgamma[c], da), w2 = mul_alone(lgamma[c], dah);
      if (within) {
        for (int m = 1; m < a.cpg; m <<= 1) {
          w1 += __shfl_xor(w1, m);
          w2 += __shfl_xor(w2, m);
        }
        if ((c & (a.cpg - 1)) == 0) use(c / a.cpg, word_of(w1, w2));
      } else {
        tot[0][c] = w1;
        tot[1][c] = w2;
      }
    });
    if (within) return;
    __syncthreads();
    each_group<NT>(r.Gb, a.cpg, [&](int c) { return f32x2_t{tot[0][c], tot[1][c]}; },
                   [&](int g, const f32x2_t& v) { use(g, word_of(v[0], v[1])); });
  };
  const auto add = [&](float (&s)[2][VEC], int j, float hh, float da) {
    s[0][j] = fmaf(da, hh, s[0][j]);
    s[1][j] += da;
  };
  float s[2][VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) s[0][j] = s[1][j] = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < n) {
      float f[VEC], d[VEC];
      vx[i].get(f);
      vd[i].get(d);
      bv.run(f, d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        add(s, j, f[j], d[j]);
        if (i >= LROWS) vda[i - LROWS][j] = d[j];
        if (FEW) vh[FEW ? i : 0][j] = f[j];
      }
      if (i < LROWS) {
#pragma unroll
        for (int j = 0; j < VEC; j += 4)
          lds_da[i][j / 4][threadIdx.x] = f32x4_t{d[j], d[j + 1], d[j + 2], d[j + 3]};
      }
    }
  }
  const double inv_n = 1.0 / ((double)a.P * a.cpg);
  const auto group = [&](int g, double x, double y) {
    g1[g] = (float)(x * inv_n);
    g2[g] = (float)(y * inv_n);
  };
  piece(
      s,
      [&](int c, float dah, float da) {
        if (!r.channel_sums) return;
        float* row = r.channel_sums + ((long long)h.u * r.W + h.w) * 2 * a.C + h.range * r.Cb;
        row[c] = dah;
        row[a.C + c] = da;
      },
      [&](int g, unsigned long long word) {
        if (!a.out) return;
        if (r.W > 1) pieces.own[g] = word;
        else group(g, word_lo(word), word_hi(word));
      });
  if (!a.out) return;
  __syncthreads();
  if (r.W > 1) {
    double s1 = 0.0, s2 = 0.0;
    const auto sum = [&](int, unsigned long long x) {
      s1 += (double)word_lo(x);
      s2 += (double)word_hi(x);
    };
    if (!pieces.collect(r, h, sum)) {
      s1 = s2 = 0.0;
      for (int w = 0; w < r.W; ++w) {
        long long fw;
        const int nw = rows_of(a, r, h, w, &fw);
        const E* px = (const E*)a.x + (at + fw) * a.x_pitch + c0;
        const E* pd = (const E*)a.dy + (at + fw) * a.dy_pitch + c0;
        const long long sx = r.ppi * a.x_pitch, sd = r.ppi * a.dy_pitch;
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[0][j] = s[1][j] = 0.0f;
#pragma unroll 1
        for (int i = 0; i < nw; ++i) {
          Held<T> x1, d1;
          x1.v = *(const u32x4_t*)(px + i * sx);
          d1.v = *(const u32x4_t*)(pd + i * sd);
          float f[VEC], d[VEC];
          x1.get(f);
          d1.get(d);
          bv.run(f, d);
#pragma unroll
          for (int j = 0; j < VEC; ++j) add(s, j, f[j], d[j]);
        }
        piece(
            s, [](int, float, float) {},
            [&](int g, unsigned long long word) { pieces.own[g] = word; });
        pieces.one(r, w, sum);
      }
    }
    pieces.join(r, s1, s2, group);
  }
  if (!h.active) return;
  float c1[VEC], c2[VEC], gam[VEC];
  GroupOf go(gl0, a.cpg);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int g = go.next(a.cpg);
    c1[j] = g1[g];
    c2[j] = g2[g];
    gam[j] = lgamma[gl0 + j];
    if (!FEW) {
      // dx = (rstd gamma) da - (rstd c2) h - rstd c1; 16-bit types: h spelt out
      // as (x - mean) rstd
      const float rs = bv.rstd[bv.at(j)];
      gam[j] = rs * gam[j];
      c2[j] = -rs * c2[j];
      c1[j] = -rs * c1[j];
      if (!T::kWide) c2[j] = rs * c2[j];
    }
  }
  E* dx = (E*)a.out + (at + first) * a.out_pitch + c0;
  const long long step = r.ppi * a.out_pitch;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < n) {
      float f[VEC], d[VEC];
      vx[i].get(f);
      if (i < LROWS) {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
          const f32x4_t q = lds_da[i][j / 4][threadIdx.x];
          d[j] = q[0];
          d[j + 1] = q[1];
          d[j + 2] = q[2];
          d[j + 3] = q[3];
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[j] = vda[i - LROWS][j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (FEW)
          f[j] = gn_dx(bv.rstd[bv.at(j)], gam[j], d[j], c1[j], vh[FEW ? i : 0][j], c2[j]);
        else
          f[j] = fmaf(d[j], gam[j],
                      fmaf(T::kWide ? bv.h(j, f[j]) : f[j] - bv.mean[bv.at(j)], c2[j], c1[j]));
      }
      Held<T> o;
      o.put(f);
      store_row<STREAM>(dx, o.v);
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
  const dim3 grid(a.units * r.NR * r.W), block(kGnResThreadsFwd);
  constexpr int R = kGnRowsFwdCompact, L = kGnRowsFwdLds;
  if (r.passes <= 4)
    hipLaunchKernelGGL((gn_resident_fwd_kernel<T, SILU, 4, 0, false, false>), grid, block, 0, s, a,
                       r);
  else if (r.compact && a.stream)
    hipLaunchKernelGGL((gn_resident_fwd_kernel<T, SILU, R, L, true, true>), grid, block, 0, s, a,
                       r);
  else if (r.compact)
    hipLaunchKernelGGL((gn_resident_fwd_kernel<T, SILU, R, L, true, false>), grid, block, 0, s, a,
                       r);
  else
    hipLaunchKernelGGL((gn_resident_fwd_kernel<T, SILU, kGnRows, 0, false, false>), grid, block, 0,
                       s, a, r);
  return (int)hipGetLastError();
}

template <class T, bool SILU, int R, int LROWS, bool COMPACT, bool STREAM>
void start_bwd(const GnTrainArgs& a, const GnResPlan& r, hipStream_t s) {
  constexpr int VEC = 16 / sizeof(typename T::store);
  const dim3 grid(a.units * r.NR * r.W), block(kGnResThreadsBwd);
  if (r.fold >= 4)
    hipLaunchKernelGGL((gn_resident_bwd_kernel<T, SILU, R, LROWS, VEC / 4, COMPACT, STREAM>), grid,
                       block, 0, s, a, r);
  else
    hipLaunchKernelGGL((gn_resident_bwd_kernel<T, SILU, R, LROWS, VEC, COMPACT, STREAM>), grid,
                       block, 0, s, a, r);
}

template <class T, bool SILU>
int run_bwd(const GnTrainArgs& a, const GnResPlan& r, hipStream_t s) {
  if (r.W > 1 && a.out) clear_words(a, r, s);
  constexpr int R = kGnRowsBwdCompact, L = kGnRowsBwdLds;
  if (r.passes <= 4) start_bwd<T, SILU, 4, 0, false, false>(a, r, s);
  else if (r.compact && a.stream) start_bwd<T, SILU, R, L, true, true>(a, r, s);
  else if (r.compact) start_bwd<T, SILU, R, L, true, false>(a, r, s);
  else start_bwd<T, SILU, kGnRows, 0, false, false>(a, r, s);
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
