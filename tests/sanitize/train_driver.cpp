// Exercises the training-side entry points' host path (checks, planning,
// workspace carving, dispatch) under AddressSanitizer and
// UndefinedBehaviorSanitizer, with host stand-ins for the launchers. The
// stand-ins check what the kernels rely on (grid and LDS limits, whole
// coverage of the channels and pixels, everything inside the workspace) and
// touch no memory; device pointers are fake, aligned and far apart. Prints
// "train driver ok" and exits 0 when every expectation holds.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "../../convolution_video_vae_amd/csrc/conv3d_train.h"
#include "../../include/conv3d.h"

static int g_fail = 0;
static int g_two_pass = 0, g_resident = 0, g_exchanged = 0, g_ns = 0;
static size_t g_ws = 0;              // workspace bytes of the call under test
static long long g_batches = 0, g_items = 0, g_blocks = 0;

static void require(bool ok, const char* what) {
  if (!ok) {
    fprintf(stderr, "stand-in launcher: %s\n", what);
    abort();
  }
}
static void* buf(int k) { return (void*)(uintptr_t)((uint64_t)(k + 1) << 42); }
static bool in_ws(const void* p, long long bytes) {
  const uintptr_t lo = (uintptr_t)buf(5);
  return (uintptr_t)p >= lo && (uintptr_t)p + (uintptr_t)bytes <= lo + g_ws;
}

namespace conv3d {

static void two_pass(const GnTrainArgs& a, bool bwd) {
  require(a.x && a.gamma && a.beta && a.stats && (bwd ? a.dy : a.out), "operands");
  require(a.chunk_px % 8 == 0 && (long long)a.chunk_px * a.chunks >= a.P &&
              (long long)a.chunk_px * (a.chunks - 1) < a.P, "chunks cover the unit");
  require((long long)a.units * a.chunks * 256 < (1LL << 32), "grid");
  require((long long)a.units * a.G * 256 < (1LL << 32), "finalize grid");
  require(in_ws(a.partial, (long long)a.units * a.chunks * a.C * 16), "partials");
  if (bwd) {
    require(in_ws(a.chan, (long long)a.units * a.C * 16), "channel sums");
    require(in_ws(a.coef, (long long)a.units * a.G * 8), "coefficients");
  }
  ++g_two_pass;
}
int launch_gn_train_fwd(const GnTrainArgs& a, void*) { two_pass(a, false); return 0; }
int launch_gn_train_bwd(const GnTrainArgs& a, void*) { two_pass(a, true); return 0; }

int launch_gn_resident(const GnTrainArgs& a, const GnResPlan& r, bool bwd, void*) {
  const int threads = bwd ? kGnResThreadsBwd : kGnResThreadsFwd, vec = 16 / elt_size(a.dtype);
  require(r.Cb == r.Vb * vec && r.Cb * r.NR == a.C && r.Gb * a.cpg == r.Cb, "whole ranges");
  require(r.Cb <= threads && r.Gb <= threads && r.ppi >= 1 && r.ppi * r.Vb <= threads, "lanes");
  require(r.piece_px == r.ppi * r.passes && (long long)r.piece_px * r.W >= a.P &&
              (long long)r.piece_px * (r.W - 1) < a.P, "pieces cover the unit");
  const int cap = !r.compact ? kGnRows : bwd ? kGnRowsBwdCompact : kGnRowsFwdCompact;
  require(r.passes >= 1 && r.passes <= cap, "rows");
  require(r.W >= 1 && r.W <= 256 && r.spin >= 0, "exchange");
  require((long long)a.units * r.NR * r.W * threads < (1LL << 32), "grid");
  const bool pow2 = (r.Vb & (r.Vb - 1)) == 0;
  require(!r.lanes || (pow2 && r.Vb <= 64 && r.ppi * r.Vb == threads), "lane exchanges");
  require(r.fold >= 1 && r.fold <= vec && a.cpg % r.fold == 0, "fold");
  require(!r.compact || (r.lanes && (bwd ? r.Cb : r.Cb / r.fold) <= kGnCompact), "compact");
  require((r.entry_lanes & (r.entry_lanes - 1)) == 0 && r.entry_lanes <= 64 &&
              r.entry_lanes * (r.Gb < threads ? 1 : r.Gb) <= threads, "entry lanes");
  if (r.W > 1) {
    require(in_ws(r.words, 8LL * a.units * r.NR * r.W * r.Gb), "words");
    ++g_exchanged;
  }
  if (r.channel_sums) {
    require(in_ws(r.channel_sums, 8LL * a.units * r.W * a.C), "channel sums");
    require(r.W == 1 || (char*)r.channel_sums >=
                            (char*)r.words + 8LL * a.units * r.NR * r.W * r.Gb, "apart");
  }
  ++g_resident;
  return 0;
}

int ns_bwd_blocks(long long M, int) { return (int)(M < 1024 ? M : 1024); }
int launch_ns_bwd(const NsBwdArgs& a, void*) {
  require(a.value && a.dy && a.gamma && a.dvalue && a.M > 0 && a.C % 8 == 0 && a.blocks > 0, "ns");
  require((!a.dgamma && !a.dbias) || in_ws(a.partial, 8LL * a.blocks * a.C), "ns partials");
  ++g_ns;
  return 0;
}

static void batch(const GradBatch& b) {
  require(b.count >= 0 && b.count <= kGradItems && b.blocks >= 0, "batch");
  int at = 0;
  for (int i = 0; i < b.count; ++i) {
    require(b.item[i].first == at && b.item[i].numel > 0 && b.item[i].src, "item");
    at += (int)((b.item[i].numel + b.chunk - 1) / b.chunk);
  }
  require(at == b.blocks && (long long)b.blocks * 256 < (1LL << 32), "blocks");
  require(in_ws(b.all, 8LL * b.partials), "partials");
  ++g_batches;
  g_items += b.count;
  g_blocks += b.blocks;
}
int launch_grad_partials(const GradBatch& b, void*) {
  batch(b);
  require(in_ws(b.partial, 8LL * b.blocks), "own partials");
  return 0;
}
int launch_grad_scale(const GradBatch& b, void*) { batch(b); return 0; }
int launch_grad_norm(const GradBatch& b, void*) { require(b.norm, "norm"); return 0; }

}  // namespace conv3d

#define EXPECT(expr, want)                                                          \
  do {                                                                              \
    const long long got_ = (long long)(expr);                                       \
    if (got_ != (long long)(want)) {                                                \
      fprintf(stderr, "%s:%d: %s = %lld, want %lld\n", __FILE__, __LINE__, #expr,   \
              got_, (long long)(want));                                             \
      ++g_fail;                                                                     \
    }                                                                               \
  } while (0)

static unsigned long long g_seed = 12345;
static unsigned rnd(unsigned n) {
  g_seed = g_seed * 6364136223846793005ull + 1442695040888963407ull;
  return (unsigned)((g_seed >> 33) % n);
}

static void gn(const conv3d_group_norm_train_desc& d, int in_place) {
  float* f[4] = {(float*)buf(1), (float*)buf(2), (float*)buf(3), (float*)buf(4)};
  const double bytes = (double)d.n * d.d * d.h * d.w * 4.0 * (2 * d.c + 70);
  if (conv3d_group_norm_train_workspace_bytes(&d, 0, &g_ws) != CONV3D_OK) {
    EXPECT(bytes > 1e12, 1);             // refused for its size alone
    return;
  }
  EXPECT(conv3d_group_norm_train_fwd(&d, buf(0), f[0], f[1], buf(6), f[2], buf(5), g_ws, nullptr),
         CONV3D_OK);
  EXPECT(conv3d_group_norm_train_workspace_bytes(&d, 1, &g_ws), CONV3D_OK);
  EXPECT(conv3d_group_norm_train_bwd(&d, buf(7), buf(0), f[0], f[1], f[2],
                                     in_place ? buf(7) : buf(6), f[3], (float*)buf(8), buf(5),
                                     g_ws, nullptr), CONV3D_OK);
  EXPECT(conv3d_group_norm_train_bwd(&d, buf(7), buf(0), f[0], f[1], f[2], nullptr, f[3], nullptr,
                                     buf(5), g_ws, nullptr), CONV3D_OK);
  EXPECT(conv3d_group_norm_train_bwd(&d, buf(7), buf(0), f[0], f[1], f[2], buf(6), nullptr,
                                     nullptr, buf(5), g_ws, nullptr), CONV3D_OK);
}

int main() {
  for (int i = 0; i < 4000; ++i) {
    conv3d_group_norm_train_desc d{};
    d.n = 1 + rnd(3);
    d.d = 1 + rnd(18);
    d.h = 1 + rnd(i % 3 ? 40 : 600);
    d.w = 1 + rnd(i % 3 ? 40 : 600);
    d.groups = 1 + rnd(i % 2 ? 40 : 300);
    d.c = d.groups * (1 + rnd(i % 5 ? 33 : 300));
    if (d.c > 65536) d.c = d.groups;
    d.t_isolated = rnd(2);
    d.silu = rnd(2);
    d.eps = 1e-5f;
    d.dtype = rnd(3);
    if (rnd(4) == 0) d.x_pitch = d.c + rnd(70);
    if (rnd(4) == 0) d.y_pitch = 2LL * d.c;
    d.dx_pitch = d.y_pitch;
    gn(d, rnd(4) == 0);
  }
  conv3d_group_norm_train_desc big = {1, 17, 256, 256, 128, 32, 1, 1, 1e-5f, CONV3D_ELT_BF16,
                                      0, 0, 0};
  const int before = g_exchanged;
  gn(big, 0);
  EXPECT(g_exchanged - before, 4);
  EXPECT(g_two_pass > 100 && g_resident > 100 && g_exchanged > 100, 1);

  EXPECT(conv3d_norm_silu_bwd_workspace_bytes(1, 5, 16, 30, 640, &g_ws), CONV3D_OK);
  EXPECT(conv3d_norm_silu_bwd(buf(0), buf(1), buf(2), 1, 5, 16, 30, 640, buf(3), buf(1),
                              (float*)buf(4), nullptr, buf(5), g_ws, nullptr), CONV3D_OK);
  EXPECT(conv3d_norm_silu_bwd(buf(0), buf(1), nullptr, 1, 5, 16, 30, 640, buf(3), buf(2), nullptr,
                              nullptr, nullptr, 0, nullptr), CONV3D_OK);
  EXPECT(g_ns, 2);

  for (int count : {0, 1, 119, 120, 121, 1000}) {
    std::vector<conv3d_grad> g((size_t)count);
    long long elements = 0;
    int full = 0;
    for (int i = 0; i < count; ++i) {
      conv3d_grad& e = g[(size_t)i];
      e.grad = (char*)buf(20) + (long long)i * (1 << 24);
      e.numel = rnd(5) == 0 ? 0 : rnd(3000000);
      e.dtype = rnd(3);
      e.out_dtype = e.dtype;
      if (rnd(2)) {
        e.out = (char*)buf(21) + (long long)(count - i) * (1 << 24);
        e.out_dtype = rnd(3);
      }
      elements += e.numel;
      full += e.numel > 0;
    }
    EXPECT(conv3d_grad_workspace_bytes(g.data(), count, &g_ws), CONV3D_OK);
    g_batches = g_items = g_blocks = 0;
    EXPECT(conv3d_grad_norm(g.data(), count, CONV3D_GRAD_NORM_L2, (float*)buf(30), buf(5), g_ws,
                            nullptr), CONV3D_OK);
    EXPECT(g_items, full);
    EXPECT(g_batches, (full + conv3d::kGradItems - 1) / conv3d::kGradItems);
    EXPECT(conv3d_grad_clip(g.data(), count, CONV3D_GRAD_NORM_INF, 1.0f, (float*)buf(30), buf(5),
                            g_ws, nullptr), CONV3D_OK);
    EXPECT(g_items, 3 * full);
    if (count > 1 && full) {
      g[0] = g[1];
      g[0].numel = g[1].numel = 10;
      g[0].out = g[1].out = nullptr;
      g[0].out_dtype = g[1].out_dtype = g[0].dtype;
      EXPECT(conv3d_grad_clip(g.data(), count, CONV3D_GRAD_NORM_L2, 1.0f, (float*)buf(30), buf(5),
                              g_ws, nullptr), CONV3D_ERR_OVERLAP);
      EXPECT(conv3d_grad_norm(g.data(), count, CONV3D_GRAD_NORM_L2, (float*)buf(30), buf(5), g_ws,
                              nullptr), CONV3D_OK);
    }
    (void)elements;
  }
  if (g_fail) return 1;
  printf("train driver ok: %d two-pass, %d resident (%d exchanged)\n", g_two_pass, g_resident,
         g_exchanged);
  return 0;
}
