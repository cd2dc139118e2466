// Arguments of the training-side kernels (GroupNorm with kept statistics and
// its backward pass, the backward pass of the channel norm + SiLU, gradient
// norm and clipping) and their launchers. Each launcher returns 0 on success
// or the HIP error code of the launch.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace conv3d {

enum EltType { ELT_BF16 = 0, ELT_FP16 = 1, ELT_FP32 = 2 };
inline int elt_size(int t) { return t == ELT_FP32 ? 4 : 2; }

// GroupNorm (conv3d_gn_train.hip). A unit is one frame (n, d) or one sample
// n: P consecutive pixels, pixel p of unit u at element (u * P + p) * pitch.
// The kernels see a unit as Q rows of V vectors of `vec` elements: a row is
// `sp` pixels (1, or for dense tensors whose channel count is no multiple of
// vec, the fewest pixels that are whole vectors).
struct GnTrainArgs {
  const void* x;
  const void* dy;            // backward only
  void* out;                 // y, or dx (null: not wanted)
  const float* gamma;        // [C]
  const float* beta;         // [C]
  float* stats;              // [units][G][2]: mean, 1/sqrt(var + eps)
  double* partial;           // [units][chunks][C][2]
  double* chan;              // backward: [units][C][2]: sum of da, of da * xhat
  float* coef;               // backward: [units][G][2]: c1, c2
  float* dgamma;             // [C] or null
  float* dbeta;              // [C] or null
  long long P;
  long long x_pitch, dy_pitch, out_pitch;   // elements
  int C, G, cpg;
  int units, chunks, chunk_px;              // chunk_px is a multiple of 8
  int dtype, silu;
  int stream;                // 1: results are stored past the caches
  float eps;
};
int launch_gn_train_fwd(const GnTrainArgs& args, void* stream);
int launch_gn_train_bwd(const GnTrainArgs& args, void* stream);

// The same with the activations read once (conv3d_gn_resident.hip): each
// work-group keeps a piece of a unit in registers. A range is Gb whole groups
// (Cb channels in Vb 16-byte vectors), NR of them make C; the unit's pixels
// are cut into W pieces of piece_px = ppi * passes.
constexpr int kGnResThreadsFwd = 512, kGnResThreadsBwd = 256;
// Rows a thread can hold: in registers alone, or in the compact form with
// some of them in the LDS that it leaves free.
constexpr int kGnRows = 12;
constexpr int kGnRowsFwdCompact = 16, kGnRowsFwdLds = 6;
constexpr int kGnRowsBwdCompact = 16, kGnRowsBwdLds = 7;
constexpr int kGnCompact = 128;                        // values of a row in the compact form
struct GnResPlan {
  int Cb, Vb, NR, Gb;
  int ppi, passes, piece_px, W;
  int lanes;                 // 1: a row is a power of two of lanes (at most a wave)
  int compact;               // 1: lanes, and at most kGnCompact channels (backward) or slots
  int fold;                  // channels of a vector that always share a group (a power of two)
  int entry_lanes;           // lanes that join one group's rows of a piece (a power of two)
  int spin;                  // polls of a thread before its work-group helps itself
  unsigned long long* words; // [units][NR][W][Gb] (W > 1)
  float* channel_sums;       // backward: [units][W][2][C], or null
};
int launch_gn_resident(const GnTrainArgs& args, const GnResPlan& plan, bool bwd, void* stream);

// Backward pass of the channel L2 norm x sqrt(C) x gamma -> SiLU
// (conv3d_ns_bwd.hip) over M rows of C channels.
struct NsBwdArgs {
  const uint16_t* value;
  const uint16_t* dy;
  const uint16_t* dskip;     // or null
  const uint16_t* gamma;
  uint16_t* dvalue;
  float* dgamma;             // or null
  float* dbias;              // or null
  float* partial;            // [blocks][2][C]
  long long M;
  int C, blocks;
};
int ns_bwd_blocks(long long M, int C);
int launch_ns_bwd(const NsBwdArgs& args, void* stream);

// Gradient norm and clipping (conv3d_grad_clip.hip).
struct GradItem {
  const void* src;
  void* dst;                 // where the clip pass writes (src: in place)
  long long numel;
  int first;                 // the first block of this tensor in its launch
  short dtype, out_dtype;
};
constexpr int kGradItems = 120;          // 32 bytes each: the arguments stay below 4 KB
struct GradBatch {
  GradItem item[kGradItems];
  double* partial;           // of this batch's first block (norm pass)
  const double* all;         // every batch's partials, or their join (clip pass)
  double* join;              // norm kernel: the join of all partials, or null
  float* norm;
  int count;                 // tensors in this batch
  int blocks;                // blocks of this batch
  int chunk;                 // elements per block
  int partials;              // of all batches
  int stream;                // 1: results are stored past the caches
  int inf;                   // the maximum of |g| instead of the 2-norm
  float max_norm;
};
static_assert(sizeof(GradBatch) <= 4096, "kernel arguments");
int launch_grad_partials(const GradBatch& batch, void* stream);
int launch_grad_norm(const GradBatch& batch, void* stream);
int launch_grad_scale(const GradBatch& batch, void* stream);

}  // namespace conv3d
