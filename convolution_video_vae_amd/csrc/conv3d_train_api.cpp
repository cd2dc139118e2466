// C-ABI of the training-side operators: argument checks, planning and
// dispatch. As in conv3d_api.cpp every check runs on the host before
// anything is enqueued.
#include <math.h>
#include <stdint.h>
#include <stdlib.h>

#include <algorithm>
#include <initializer_list>
#include <vector>

#include "../../include/conv3d.h"
#include "conv3d_checks.h"
#include "conv3d_train.h"

using namespace conv3d;

namespace {

bool aligned_to(const void* p, int bytes) { return ((uintptr_t)p % (unsigned)bytes) == 0; }
bool elt_ok(int t) { return t == CONV3D_ELT_BF16 || t == CONV3D_ELT_FP16 || t == CONV3D_ELT_FP32; }

// Results of more bytes are stored past the caches: half of the memory-side one.
constexpr long long kStreamBytes = 128LL << 20;

// ------------------------------------------------------------- GroupNorm

constexpr long long kGnMaxItems = (1LL << 24) - 1;   // work-groups of one launch (grid x 256 < 2^32)
constexpr long long kGnTarget = 2048;                // work-groups a pass aims at
constexpr long long kGnMinChunk = 64;                // pixels; a chunk leaves 16 bytes per channel

struct GnTrainPlan {
  GnTrainArgs a;
  size_t off_chan, off_coef, total;
  bool fits;                 // r: the activations may stay in registers
  GnResPlan r;
  size_t off_sums;
};

// Pieces of one exchange: half of the 512 work-groups that the chip holds, so
// that two calls side by side still find room. (Resident against two passes,
// backward: [1,8,256,512,128] bf16, 256 pieces, 206 and 257 us; at 384 pieces,
// [1,4,384,512,128], 182 and 197 us, left to two passes for that room.)
constexpr int kGnMaxPieces = 256;
constexpr int kGnFill = 256;             // work-groups that give every CU one
// Rows per thread up to which one work-group per narrow range is better than
// an exchange, where the chip is not filled ([1,5,32,32,512] bf16 forward, 8
// rows: 10.6 and 11.9 us; backward, 16 rows: 19.4 and 15.2 us).
constexpr int kGnAloneRows = 10;
constexpr int kGnSpin = 5000;            // polls (some 5 ms) before a work-group helps itself

// CONV3D_GN_SPIN: another bound, for tests (0: no work-group waits, each forms
// the sums of its unit's other pieces itself).
int spin_bound() {
  const char* e = getenv("CONV3D_GN_SPIN");
  if (!e) return kGnSpin;
  const long v = strtol(e, nullptr, 10);
  return (int)std::min(std::max(v, 0L), (long)kGnSpin);
}

// Time of n work-groups of `passes` rows per thread in W pieces per range, in
// tenths of a microsecond, as measured: a work-group takes 8 us and 0.6 us a
// row where it has its CU alone, 9 us and 1 us beside another; 512 of them are
// resident, and up to 1024 take two whole rounds; the exchange takes 3 us.
// ([1,17,64,64,256] bf16 forward: 272, 408, 544 and 816 work-groups of 16, 11,
// 8 and 6 rows take 29, 24, 33 and 29 us. Over 44 shapes the number of pieces
// of least such time is 2.4% faster forward and 1.4% backward than the smallest
// that gives 256 work-groups: between 17% faster and 3% slower.)
long long piece_cost(long long n, long long passes, long long W) {
  const long long exchange = W > 1 ? 30 : 0;
  if (n <= kGnFill) return 80 + 6 * passes + exchange;
  const long long each = 90 + 10 * passes;
  if (n <= 4 * kGnFill) return (n + 2 * kGnFill - 1) / (2 * kGnFill) * each + exchange;
  return (n + kGnFill) * each / (2 * kGnFill) + exchange;
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Ranges and pieces of the resident form for 16-byte vectors; false where a
// unit's pieces are too many to be on the chip together.
bool plan_resident(const GnTrainArgs& a, bool bwd, GnResPlan* r) {
  const int size = elt_size(a.dtype), vec = 16 / size;
  int rows = 0;                          // a thread can hold
  const int threads = bwd ? kGnResThreadsBwd : kGnResThreadsFwd;
  if (a.C % vec) return false;
  const int quantum = a.cpg / gcd(a.cpg, vec) * vec;    // whole groups in whole vectors
  const auto lay = [&](int Cb) {
    r->Cb = Cb;
    r->Vb = Cb / vec;
    r->NR = a.C / Cb;
    r->Gb = Cb / a.cpg;
    r->ppi = threads / r->Vb;
    r->lanes = r->Vb <= 64 && (r->Vb & (r->Vb - 1)) == 0;
    r->fold = 1;
    while (r->fold < vec && a.cpg % (2 * r->fold) == 0) r->fold *= 2;
    r->compact = r->lanes && (bwd ? Cb : Cb / r->fold) <= kGnCompact;
    rows = !r->compact ? kGnRows : bwd ? kGnRowsBwdCompact : kGnRowsFwdCompact;
    const int entries = (r->lanes ? threads / 64 : r->ppi) * (a.cpg / r->fold);
    r->entry_lanes = 1;
    while (r->entry_lanes < 32 && 2 * r->entry_lanes <= entries &&
           2 * r->entry_lanes * r->Gb <= threads)
      r->entry_lanes *= 2;
  };
  const int limit = std::min(a.C, threads);
  // few units: one work-group per range, the narrowest of at least 64 bytes a
  // pixel. (Where such ranges fill the chip, half lines cost more than an
  // exchange: [8,5,32,32,512] bf16 forward 39.5 us, as below 26.7 us.)
  for (int Cb = quantum; Cb <= limit; Cb += quantum) {
    if (a.C % Cb || (Cb * size < 64 && Cb < a.C)) continue;
    lay(Cb);
    const long long passes = (a.P + r->ppi - 1) / r->ppi;
    if (passes > kGnAloneRows || (long long)a.units * r->NR > kGnFill) break;
    r->passes = (int)passes;
    r->W = 1;
    r->piece_px = r->ppi * r->passes;
    return true;
  }
  // pieces of ranges of whole 128-byte lines: the number that piece_cost finds
  // best among those that hold the unit
  for (int Cb = quantum; Cb <= limit; Cb += quantum) {
    if (a.C % Cb || (Cb * size < 128 && Cb < a.C)) continue;
    lay(Cb);
    const long long lanes = (a.P + r->ppi - 1) / r->ppi;        // rows per thread in all
    const long long ranges = (long long)a.units * r->NR;
    const long long fewest = (lanes + rows - 1) / rows;
    if (fewest > kGnMaxPieces) return false;
    const long long most = std::min((long long)kGnMaxPieces, std::max(fewest, (lanes + 1) / 2));
    long long best = fewest;
    for (long long W = fewest; W <= most; ++W)
      if (piece_cost(ranges * W, (lanes + W - 1) / W, W) <
          piece_cost(ranges * best, (lanes + best - 1) / best, best))
        best = W;
    r->passes = (int)((lanes + best - 1) / best);
    r->piece_px = r->ppi * r->passes;
    r->W = (int)((a.P + r->piece_px - 1) / r->piece_px);
    return (long long)a.units * r->NR * r->W <= kGnMaxItems / 2 &&
           (long long)a.units * r->NR * r->W * r->Gb <= (1LL << 30);
  }
  return false;
}

conv3d_status plan_gn_train(const conv3d_group_norm_train_desc* d, bool bwd, GnTrainPlan* pl) {
  if (!d) return CONV3D_ERR_NULL;
  if (d->n <= 0 || d->d <= 0 || d->h <= 0 || d->w <= 0 || d->c <= 0 || d->groups <= 0)
    return CONV3D_ERR_SHAPE;
  if (!(d->eps > 0.0f) || !isfinite(d->eps)) return CONV3D_ERR_SHAPE;
  if (d->c % d->groups) return CONV3D_ERR_SHAPE;
  if (!elt_ok(d->dtype)) return CONV3D_ERR_UNSUPPORTED;
  const long long xp = d->x_pitch ? d->x_pitch : d->c, yp = d->y_pitch ? d->y_pitch : d->c;
  const long long dp = d->dx_pitch ? d->dx_pitch : d->c;
  if (xp < d->c || yp < d->c || dp < d->c) return CONV3D_ERR_SHAPE;
  if (d->c > 65536) return CONV3D_ERR_UNSUPPORTED;
  const long long units = d->t_isolated ? prod({d->n, d->d}) : d->n;
  const long long P = prod({d->t_isolated ? 1LL : (long long)d->d, d->h, d->w});
  const int size = elt_size(d->dtype);
  if (prod({units, P, std::max(xp, std::max(yp, dp)), size}) > (1LL << 40))
    return CONV3D_ERR_UNSUPPORTED;
  const long long want = std::max(1LL, (kGnTarget + units - 1) / units);
  long long chunk = std::max((P + want - 1) / want, std::min(kGnMinChunk, P));
  chunk = (chunk + 7) / 8 * 8;
  const long long chunks = (P + chunk - 1) / chunk;
  if (prod({units, chunks}) > kGnMaxItems || prod({units, d->groups}) > kGnMaxItems ||
      chunk > (1LL << 30))
    return CONV3D_ERR_UNSUPPORTED;
  GnTrainArgs& a = pl->a;
  a = GnTrainArgs{};
  a.P = P;
  a.C = d->c;
  a.G = d->groups;
  a.cpg = d->c / d->groups;
  a.x_pitch = xp;
  a.dy_pitch = yp;
  a.out_pitch = bwd ? dp : yp;
  a.units = (int)units;
  a.chunks = (int)chunks;
  a.chunk_px = (int)chunk;
  a.dtype = d->dtype;
  a.silu = d->silu ? 1 : 0;
  a.stream = prod({units, P, a.C, size}) > kStreamBytes;
  a.eps = d->eps;
  size_t at = (size_t)units * chunks * a.C * 16;
  pl->off_chan = at = (at + 255) / 256 * 256;
  if (bwd) {
    at += (size_t)units * a.C * 16;
    pl->off_coef = at = (at + 255) / 256 * 256;
    at += (size_t)units * a.G * 8;
  }
  pl->total = (at + 255) / 256 * 256;
  // the resident form needs its words and channel sums instead
  pl->r = GnResPlan{};
  pl->r.spin = spin_bound();
  pl->fits = plan_resident(a, bwd, &pl->r);
  if (pl->fits) {
    const GnResPlan& r = pl->r;
    at = r.W > 1 ? (size_t)units * r.NR * r.W * r.Gb * 8 : 0;
    pl->off_sums = at = (at + 255) / 256 * 256;
    if (bwd) at += (size_t)units * r.W * 2 * a.C * 4;
    pl->total = std::max(pl->total, (at + 255) / 256 * 256);
  }
  return CONV3D_OK;
}

// Whether an operand's pixels are 16-byte vectors.
bool vectors(const void* p, long long pitch, int size) {
  return aligned16(p) && (pitch * size) % 16 == 0;
}

// One operand: `pixels` rows of `c` elements at a pitch.
struct Pitched {
  Range r;
  long long row, pitch;   // bytes
};

Pitched pitched(const void* p, long long pixels, int c, long long pitch, int size) {
  return {range_of(p, ((pixels - 1) * pitch + c) * size), (long long)c * size, pitch * size};
}

// Whether two operands share memory. Two channel slices of one wider buffer
// (equal pitches) are told apart although their ranges interleave.
bool share(const Pitched& a, const Pitched& b) {
  if (!overlaps(a.r, b.r)) return false;
  if (a.pitch != b.pitch) return true;
  const long long d = (long long)((b.r.lo - a.r.lo) % (uintptr_t)a.pitch);
  const long long off = b.r.lo >= a.r.lo ? d : (a.pitch - (long long)((a.r.lo - b.r.lo) % (uintptr_t)a.pitch)) % a.pitch;
  return off < a.row || off + b.row > a.pitch;
}

}  // namespace

extern "C" {

conv3d_status conv3d_group_norm_train_workspace_bytes(const conv3d_group_norm_train_desc* desc,
                                                      int backward, size_t* bytes) {
  if (!bytes) return CONV3D_ERR_NULL;
  GnTrainPlan pl;
  const conv3d_status st = plan_gn_train(desc, backward != 0, &pl);
  if (st != CONV3D_OK) return st;
  *bytes = pl.total;
  return CONV3D_OK;
}

conv3d_status conv3d_group_norm_train_fwd(const conv3d_group_norm_train_desc* desc, const void* x,
                                          const float* gamma, const float* beta, void* y,
                                          float* stats, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  if (!desc || !x || !gamma || !beta || !y || !stats) return CONV3D_ERR_NULL;
  GnTrainPlan pl;
  const conv3d_status st = plan_gn_train(desc, false, &pl);
  if (st != CONV3D_OK) return st;
  GnTrainArgs& a = pl.a;
  const int size = elt_size(a.dtype);
  if (!aligned_to(x, size) || !aligned_to(y, size) || !aligned_to(gamma, 4) ||
      !aligned_to(beta, 4) || !aligned_to(stats, 4))
    return CONV3D_ERR_ALIGN;
  if (!workspace || workspace_bytes < pl.total) return CONV3D_ERR_WORKSPACE;
  if (!aligned16(workspace)) return CONV3D_ERR_ALIGN;
  const long long pixels = a.units * a.P;
  const Pitched px = pitched(x, pixels, a.C, a.x_pitch, size);
  const Pitched py = pitched(y, pixels, a.C, a.out_pitch, size);
  const Range rg = range_of(gamma, 4LL * a.C), rb = range_of(beta, 4LL * a.C);
  const Range rs = range_of(stats, 8LL * a.units * a.G);
  const Range rw = range_of(workspace, (long long)pl.total);
  if (share(px, py)) return CONV3D_ERR_OVERLAP;
  for (const Range& o : {rs, rw})
    for (const Range& i : {px.r, py.r, rg, rb})
      if (overlaps(o, i)) return CONV3D_ERR_OVERLAP;
  if (overlaps(rs, rw) || overlaps(py.r, rg) || overlaps(py.r, rb)) return CONV3D_ERR_OVERLAP;
  a.x = x;
  a.out = y;
  a.gamma = gamma;
  a.beta = beta;
  a.stats = stats;
  if (pl.fits && vectors(x, a.x_pitch, size) && vectors(y, a.out_pitch, size)) {
    pl.r.words = (unsigned long long*)workspace;
    return launch_gn_resident(a, pl.r, false, stream) ? CONV3D_ERR_HIP : CONV3D_OK;
  }
  a.partial = (double*)workspace;
  return launch_gn_train_fwd(a, stream) ? CONV3D_ERR_HIP : CONV3D_OK;
}

conv3d_status conv3d_group_norm_train_bwd(const conv3d_group_norm_train_desc* desc, const void* dy,
                                          const void* x, const float* gamma, const float* beta,
                                          const float* stats, void* dx, float* dgamma,
                                          float* dbeta, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  if (!desc || !dy || !x || !gamma || !beta || !stats) return CONV3D_ERR_NULL;
  if (!dx && !dgamma && !dbeta) return CONV3D_ERR_NULL;
  GnTrainPlan pl;
  const conv3d_status st = plan_gn_train(desc, true, &pl);
  if (st != CONV3D_OK) return st;
  GnTrainArgs& a = pl.a;
  const int size = elt_size(a.dtype);
  if (!aligned_to(x, size) || !aligned_to(dy, size) || !aligned_to(dx, size) ||
      !aligned_to(gamma, 4) || !aligned_to(beta, 4) || !aligned_to(stats, 4) ||
      !aligned_to(dgamma, 4) || !aligned_to(dbeta, 4))
    return CONV3D_ERR_ALIGN;
  if (!workspace || workspace_bytes < pl.total) return CONV3D_ERR_WORKSPACE;
  if (!aligned16(workspace)) return CONV3D_ERR_ALIGN;
  const long long pixels = a.units * a.P;
  const Pitched px = pitched(x, pixels, a.C, a.x_pitch, size);
  const Pitched pd = pitched(dy, pixels, a.C, a.dy_pitch, size);
  const Range ins[] = {px.r, pd.r, range_of(gamma, 4LL * a.C), range_of(beta, 4LL * a.C),
                       range_of(stats, 8LL * a.units * a.G)};
  const Range small[] = {range_of(dgamma, 4LL * a.C), range_of(dbeta, 4LL * a.C),
                         range_of(workspace, (long long)pl.total)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : ins)
      if (overlaps(small[i], r)) return CONV3D_ERR_OVERLAP;
    for (int j = 0; j < i; ++j)
      if (overlaps(small[i], small[j])) return CONV3D_ERR_OVERLAP;
  }
  bool in_place = false;
  if (dx) {
    const Pitched po = pitched(dx, pixels, a.C, a.out_pitch, size);
    in_place = dx == dy && a.out_pitch == a.dy_pitch;
    if (share(po, px) || (!in_place && share(po, pd))) return CONV3D_ERR_OVERLAP;
    for (const Range& r : small)
      if (overlaps(po.r, r)) return CONV3D_ERR_OVERLAP;
    for (int i = 2; i < 5; ++i)
      if (overlaps(po.r, ins[i])) return CONV3D_ERR_OVERLAP;
  }
  a.x = x;
  a.dy = dy;
  a.out = dx;
  a.gamma = gamma;
  a.beta = beta;
  a.stats = const_cast<float*>(stats);
  a.partial = (double*)workspace;
  a.chan = (double*)((char*)workspace + pl.off_chan);
  a.coef = (float*)((char*)workspace + pl.off_coef);
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  // in place, a work-group that has to form another piece's sums itself would
  // read what that piece's own work-group may have overwritten
  if (pl.fits && !(in_place && pl.r.W > 1) && vectors(x, a.x_pitch, size) &&
      vectors(dy, a.dy_pitch, size) && (!dx || vectors(dx, a.out_pitch, size))) {
    pl.r.words = (unsigned long long*)workspace;
    pl.r.channel_sums =
        dgamma || dbeta ? (float*)((char*)workspace + pl.off_sums) : nullptr;
    return launch_gn_resident(a, pl.r, true, stream) ? CONV3D_ERR_HIP : CONV3D_OK;
  }
  return launch_gn_train_bwd(a, stream) ? CONV3D_ERR_HIP : CONV3D_OK;
}

// ------------------------------------------------- channel norm + SiLU, backward

static conv3d_status ns_bwd_check(int n, int d, int h, int w, int c, long long* M,
                                  long long* bytes, size_t* ws) {
  if (n <= 0 || d <= 0 || h <= 0 || w <= 0 || c <= 0) return CONV3D_ERR_SHAPE;
  if (c % 8) return CONV3D_ERR_ALIGN;
  if (c > 2048) return CONV3D_ERR_UNSUPPORTED;
  *M = prod({n, d, h, w});
  *bytes = prod({*M, c, 2});
  if (*bytes > (1LL << 40)) return CONV3D_ERR_UNSUPPORTED;
  *ws = ((size_t)ns_bwd_blocks(*M, c) * 2 * c * 4 + 255) / 256 * 256;
  return CONV3D_OK;
}

conv3d_status conv3d_norm_silu_bwd_workspace_bytes(int n, int d, int h, int w, int c,
                                                   size_t* bytes) {
  if (!bytes) return CONV3D_ERR_NULL;
  long long M, t;
  return ns_bwd_check(n, d, h, w, c, &M, &t, bytes);
}

conv3d_status conv3d_norm_silu_bwd(const void* value, const void* dy, const void* dskip, int n,
                                   int d, int h, int w, int c, const void* gamma, void* dvalue,
                                   float* dgamma, float* dbias, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (!value || !dy || !gamma || !dvalue) return CONV3D_ERR_NULL;
  long long M, bytes;
  size_t ws;
  const conv3d_status st = ns_bwd_check(n, d, h, w, c, &M, &bytes, &ws);
  if (st != CONV3D_OK) return st;
  if (!aligned16(value) || !aligned16(dy) || !aligned16(dskip) || !aligned16(gamma) ||
      !aligned16(dvalue) || !aligned_to(dgamma, 4) || !aligned_to(dbias, 4))
    return CONV3D_ERR_ALIGN;
  const bool sums = dgamma || dbias;
  if (sums && (!workspace || workspace_bytes < ws)) return CONV3D_ERR_WORKSPACE;
  if (sums && !aligned16(workspace)) return CONV3D_ERR_ALIGN;
  const Range rv = range_of(value, bytes), ry = range_of(dy, bytes), rs = range_of(dskip, bytes);
  const Range rg = range_of(gamma, 2LL * c), ro = range_of(dvalue, bytes);
  const Range outs[] = {ro, range_of(dgamma, 4LL * c), range_of(dbias, 4LL * c),
                        sums ? range_of(workspace, (long long)ws) : Range()};
  for (int i = 0; i < 4; ++i) {
    const bool big = i == 0;
    if (overlaps(outs[i], rv) || overlaps(outs[i], rg) ||
        (!(big && dvalue == dy) && overlaps(outs[i], ry)) ||
        (!(big && dvalue == dskip) && overlaps(outs[i], rs)))
      return CONV3D_ERR_OVERLAP;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return CONV3D_ERR_OVERLAP;
  }
  NsBwdArgs a{};
  a.value = (const uint16_t*)value;
  a.dy = (const uint16_t*)dy;
  a.dskip = (const uint16_t*)dskip;
  a.gamma = (const uint16_t*)gamma;
  a.dvalue = (uint16_t*)dvalue;
  a.dgamma = dgamma;
  a.dbias = dbias;
  a.partial = (float*)workspace;
  a.M = M;
  a.C = c;
  a.blocks = ns_bwd_blocks(M, c);
  return launch_ns_bwd(a, stream) ? CONV3D_ERR_HIP : CONV3D_OK;
}

}  // extern "C"

// ------------------------------------------------------ gradient norm and clipping

namespace {

constexpr int kGradMaxCount = 1 << 20;
constexpr long long kGradMaxElements = 1LL << 40;

struct GradPlan {
  long long chunk = 0;         // elements per work-group
  long long partials = 0;      // work-groups over all tensors
  size_t bytes = 0;
};

// Elements per work-group. Each work-group leaves one partial, and each one of
// the clip pass adds all partials (an encoder's 167 M gradients: 282 us with
// 1024 work-groups, 278 us with 2000; 34 M that need no clipping: 20 and 23 us).
constexpr long long kGradMinChunk = 4096, kGradMidChunk = 32768, kGradStep = 2048;
long long grad_chunk(long long total) {
  const long long few = total / 1024, many = std::max(kGradMidChunk, total / 2000);
  return std::max(kGradMinChunk, (std::min(few, many) + kGradStep) / kGradStep * kGradStep);
}

// Partials up to which every work-group of the clip pass adds them by itself:
// more than large tensors leave (some 2000). Of more, a launch between the
// passes adds them once (n tensors of 64 values, one partial each, by
// themselves and by a launch: 500 33 and 34 us, 2000 107 and 95, 4000 234 and
// 181, 32000 4822 and 1360).
constexpr long long kGradDirect = 2560;

long long grad_blocks(long long numel, long long chunk) { return (numel + chunk - 1) / chunk; }

conv3d_status plan_grads(const conv3d_grad* g, int count, GradPlan* pl) {
  if (count < 0) return CONV3D_ERR_SHAPE;
  if (count > 0 && !g) return CONV3D_ERR_NULL;
  if (count > kGradMaxCount) return CONV3D_ERR_UNSUPPORTED;
  long long total = 0;
  for (int i = 0; i < count; ++i) {
    if (g[i].numel < 0) return CONV3D_ERR_SHAPE;
    if (!elt_ok(g[i].dtype) || !elt_ok(g[i].out_dtype)) return CONV3D_ERR_UNSUPPORTED;
    if (g[i].numel > kGradMaxElements || (total += g[i].numel) > kGradMaxElements)
      return CONV3D_ERR_UNSUPPORTED;
  }
  pl->chunk = grad_chunk(total);
  for (int i = 0; i < count; ++i) pl->partials += grad_blocks(g[i].numel, pl->chunk);
  if (pl->chunk > (1LL << 30) || pl->partials > (1LL << 24) - 1) return CONV3D_ERR_UNSUPPORTED;
  // the partials, and behind them their join
  pl->bytes = ((size_t)(pl->partials + 1) * 8 + 255) / 256 * 256;
  return CONV3D_OK;
}

struct Span {
  uintptr_t lo, hi;
};

// By address; lists that come in that order already, as most do, are not sorted.
void by_address(std::vector<Span>& v) {
  const auto less = [](const Span& a, const Span& b) { return a.lo < b.lo; };
  if (!std::is_sorted(v.begin(), v.end(), less)) std::sort(v.begin(), v.end(), less);
}

// Every written range must lie apart from every other range.
bool spans_clash(std::vector<Span>& reads, std::vector<Span>& writes) {
  by_address(reads);
  by_address(writes);
  size_t i = 0;
  uintptr_t read_to = 0;                 // the end of all reads that begin below w.hi
  for (size_t k = 0; k < writes.size(); ++k) {
    const Span& w = writes[k];
    if (k && w.lo < writes[k - 1].hi) return true;
    for (; i < reads.size() && reads[i].lo < w.hi; ++i) read_to = std::max(read_to, reads[i].hi);
    if (read_to > w.lo) return true;
  }
  return false;
}

conv3d_status run_grads(const conv3d_grad* g, int count, int norm_type, bool clip, float max_norm,
                        float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  if (norm_type != CONV3D_GRAD_NORM_L2 && norm_type != CONV3D_GRAD_NORM_INF)
    return CONV3D_ERR_UNSUPPORTED;
  if (clip && (!(max_norm >= 0.0f) || !isfinite(max_norm))) return CONV3D_ERR_SHAPE;
  if (!norm) return CONV3D_ERR_NULL;
  GradPlan pl;
  conv3d_status st = plan_grads(g, count, &pl);
  if (st != CONV3D_OK) return st;
  std::vector<Span> reads, writes;
  reads.reserve((size_t)count);
  writes.reserve((size_t)count + 2);
  int last = -1;                         // the last tensor that holds anything
  long long out_bytes = 0;
  for (int i = 0; i < count; ++i) {
    if (g[i].numel == 0) continue;
    last = i;
    const uintptr_t src = (uintptr_t)g[i].grad;
    if (!src) return CONV3D_ERR_NULL;
    if (src % (unsigned)elt_size(g[i].dtype)) return CONV3D_ERR_ALIGN;
    out_bytes += g[i].numel * elt_size(g[i].out_dtype);
    const bool in_place = !g[i].out || g[i].out == g[i].grad;
    if (clip && in_place && g[i].out_dtype != g[i].dtype) return CONV3D_ERR_OVERLAP;
    (clip && in_place ? writes : reads)
        .push_back({src, src + (uintptr_t)g[i].numel * elt_size(g[i].dtype)});
    if (clip && !in_place) {
      const uintptr_t dst = (uintptr_t)g[i].out;
      if (dst % (unsigned)elt_size(g[i].out_dtype)) return CONV3D_ERR_ALIGN;
      writes.push_back({dst, dst + (uintptr_t)g[i].numel * elt_size(g[i].out_dtype)});
    }
  }
  if (!aligned_to(norm, 4)) return CONV3D_ERR_ALIGN;
  if (!workspace || workspace_bytes < pl.bytes) return CONV3D_ERR_WORKSPACE;
  if (!aligned16(workspace)) return CONV3D_ERR_ALIGN;
  writes.push_back({(uintptr_t)norm, (uintptr_t)norm + 4});
  writes.push_back({(uintptr_t)workspace, (uintptr_t)workspace + pl.bytes});
  if (spans_clash(reads, writes)) return CONV3D_ERR_OVERLAP;

  double* partial = (double*)workspace;
  GradBatch b{};
  b.all = partial;
  b.norm = norm;
  b.chunk = (int)pl.chunk;
  b.partials = (int)pl.partials;
  b.stream = out_bytes > kStreamBytes;
  b.inf = norm_type == CONV3D_GRAD_NORM_INF;
  b.max_norm = max_norm;
  for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
    b.partial = partial;
    b.norm = norm;
    b.count = b.blocks = 0;
    if (pass == 1 && pl.partials > kGradDirect) {
      b.join = partial + pl.partials;
      if (launch_grad_norm(b, stream)) return CONV3D_ERR_HIP;
      b.all = b.join;
      b.partials = 1;
      b.norm = nullptr;
    }
    for (int i = 0; i < count; ++i) {
      if (g[i].numel == 0) continue;
      GradItem& it = b.item[b.count++];
      it.src = g[i].grad;
      it.dst = g[i].out ? g[i].out : g[i].grad;
      it.numel = g[i].numel;
      it.first = b.blocks;
      it.dtype = (short)g[i].dtype;
      it.out_dtype = (short)g[i].out_dtype;
      b.blocks += (int)grad_blocks(g[i].numel, pl.chunk);
      if (b.count < kGradItems && i != last) continue;
      if (pass == 0 ? launch_grad_partials(b, stream) : launch_grad_scale(b, stream))
        return CONV3D_ERR_HIP;
      b.partial += b.blocks;
      b.norm = nullptr;                  // the first batch of the clip pass writes it
      b.count = b.blocks = 0;
    }
  }
  if (!clip || pl.partials == 0) {
    b.norm = norm;
    if (launch_grad_norm(b, stream)) return CONV3D_ERR_HIP;
  }
  return CONV3D_OK;
}

}  // namespace

extern "C" {

conv3d_status conv3d_grad_workspace_bytes(const conv3d_grad* grads, int count, size_t* bytes) {
  if (!bytes) return CONV3D_ERR_NULL;
  GradPlan pl;
  const conv3d_status st = plan_grads(grads, count, &pl);
  if (st != CONV3D_OK) return st;
  *bytes = pl.bytes;
  return CONV3D_OK;
}

conv3d_status conv3d_grad_norm(const conv3d_grad* grads, int count, int norm_type, float* norm,
                               void* workspace, size_t workspace_bytes, void* stream) try {
  return run_grads(grads, count, norm_type, false, 0.0f, norm, workspace, workspace_bytes, stream);
} catch (...) {            // the host's memory is exhausted
  return CONV3D_ERR_UNSUPPORTED;
}

conv3d_status conv3d_grad_clip(const conv3d_grad* grads, int count, int norm_type, float max_norm,
                               float* norm, void* workspace, size_t workspace_bytes,
                               void* stream) try {
  return run_grads(grads, count, norm_type, true, max_norm, norm, workspace, workspace_bytes,
                   stream);
} catch (...) {
  return CONV3D_ERR_UNSUPPORTED;
}

}  // extern "C"
