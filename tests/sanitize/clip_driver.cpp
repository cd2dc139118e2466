// Long gradient lists through conv3d_grad_clip, with host stand-ins for the
// launchers: what the clip pass's work-groups add is bounded whatever the
// number of tensors. Prints "clip driver ok" and exits 0.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "../../convolution_video_vae_amd/csrc/conv3d_train.h"
#include "../../include/conv3d.h"

static size_t g_ws = 0;
static long long g_added = 0, g_partials = 0, g_joined = 0;
static int g_norms = 0;

static void require(bool ok, const char* what) {
  if (!ok) {
    fprintf(stderr, "clip driver: %s\n", what);
    exit(1);
  }
}
static char* ws() { return (char*)(uintptr_t)(1ULL << 45); }
static bool in_ws(const void* p, long long bytes) {
  return (char*)p >= ws() && (char*)p + bytes <= ws() + g_ws;
}

namespace conv3d {
int launch_gn_train_fwd(const GnTrainArgs&, void*) { return 1; }
int launch_gn_train_bwd(const GnTrainArgs&, void*) { return 1; }
int launch_gn_resident(const GnTrainArgs&, const GnResPlan&, bool, void*) { return 1; }
int ns_bwd_blocks(long long, int) { return 1; }
int launch_ns_bwd(const NsBwdArgs&, void*) { return 1; }
int launch_grad_partials(const GradBatch& b, void*) {
  require(in_ws(b.partial, 8LL * b.blocks), "partials in the workspace");
  g_partials += b.blocks;
  return 0;
}
int launch_grad_norm(const GradBatch& b, void*) {
  require(b.norm && in_ws(b.all, 8LL * b.partials), "operands of the norm");
  require(b.partials == g_partials, "all partials are there");
  if (b.join) {
    require(in_ws(b.join, 8) && b.join >= b.all + b.partials, "the join lies behind the partials");
    g_joined = b.partials;
  }
  ++g_norms;
  return 0;
}
int launch_grad_scale(const GradBatch& b, void*) {
  require(in_ws(b.all, 8LL * b.partials), "sums in the workspace");
  require(b.partials == g_partials || (b.partials == 1 && g_joined == g_partials), "all are added");
  require((b.norm != nullptr) == (g_norms == 0), "the norm is written once");
  if (b.norm) ++g_norms;
  g_added += (long long)b.blocks * b.partials;
  return 0;
}
}  // namespace conv3d

int main() {
  float* norm = (float*)(uintptr_t)(1ULL << 44);
  for (int count : {1, 73, 2560, 2561, 100000, 1 << 20}) {
    for (int numel : {1, 700}) {
      std::vector<conv3d_grad> g((size_t)count);
      for (int i = 0; i < count; ++i)
        g[(size_t)i] = {(void*)(uintptr_t)((1ULL << 40) + 4096ULL * i), nullptr, numel,
                        CONV3D_ELT_FP32, CONV3D_ELT_FP32};
      require(conv3d_grad_workspace_bytes(g.data(), count, &g_ws) == CONV3D_OK, "workspace");
      g_added = g_partials = g_joined = g_norms = 0;
      require(conv3d_grad_clip(g.data(), count, CONV3D_GRAD_NORM_L2, 1.0f, norm, ws(), g_ws,
                               nullptr) == CONV3D_OK, "clip");
      require(g_partials == count && g_norms == 1, "one norm of all");
      printf("%d tensors: %lld partials added in the clip pass\n", count, g_added);
      require(g_added <= 8192LL * count, "work in proportion to the list");
      g_partials = g_norms = 0;
      require(conv3d_grad_norm(g.data(), count, CONV3D_GRAD_NORM_L2, norm, ws(), g_ws, nullptr) ==
                  CONV3D_OK && g_norms == 1, "norm");
    }
  }
  printf("clip driver ok\n");
  return 0;
}
