// Drives the drafter-training entry points' host layer (spec_train_api.hip) with the kernel
// launchers replaced by stand-ins, built for the CPU under AddressSanitizer and
// UndefinedBehaviorSanitizer: every array carved from a workspace of exactly the reported size is
// checked and cleared, refusals must return their code before any launch.
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "host_stubs.h"
#include "spec_device.h"
#include "spec_train.h"
#include "spec_verify.h"

using hoststub::carved;

namespace specv {

hipError_t launch_row_topk(const TopkArgs& a, int, hipStream_t) {
  ++hoststub::g_launches;
  const size_t n = (size_t)a.R * a.n_seg;
  carved("candidates", a.cand, n * a.cap * sizeof(uint64_t));
  carved("candidate counts", a.n_cand, n * sizeof(int32_t));
  carved("segment sums", a.ms, n * kWaves * sizeof(MaxSum));
  if (a.cap < a.K || (a.cap & (a.cap - 1)) || a.seg > kTrSeg || a.seg % 8 || (int64_t)a.n_seg * a.seg < a.V) ++hoststub::g_errors;
  return hipSuccess;
}
hipError_t launch_topk_distill(const DistillArgs& a, int, hipStream_t) {
  ++hoststub::g_launches;
  carved("segment sums", a.ms, (size_t)a.R * a.n_seg * kWaves * sizeof(MaxSum));
  if (a.d_logits) {
    carved("row factors", a.rows, (size_t)a.R * sizeof(DistillRow));
    carved("list gradients", a.d_list, (size_t)a.R * a.K * sizeof(float));
  }
  return hipSuccess;
}
hipError_t launch_head_loss(const HlArgs& a, hipStream_t) {
  ++hoststub::g_launches;
  const HlPlan& p = a.plan;
  carved("tile records", a.rec, (size_t)p.n_ct * p.n_wave * p.Rp * sizeof(float2));
  carved("target logits", a.ly, (size_t)p.Rp * sizeof(float));
  carved("rows", a.rows, (size_t)p.Rp * sizeof(HlRow));
  if (p.bn < 64 || p.bn > 256 || p.bn % 32 || (p.bn > 64 && p.bn < 128)) ++hoststub::g_errors;
  if (p.Rp < a.R || p.Rp % kHlDepth || p.piece % kHlTile || p.piece <= 0 || p.n_split < 1) ++hoststub::g_errors;
  // a piece's gradient stays within 256 MB, or one tile's columns
  if (p.piece > kHlTile && (int64_t)p.Rp * p.piece * 2 > ((int64_t)1 << 28)) ++hoststub::g_errors;
  if (a.d_hidden || a.d_weight) {
    carved("hidden copy", a.hz, (size_t)p.Rp * a.D * sizeof(uint16_t));
    carved("logit gradients", a.g, (size_t)p.Rp * p.piece * sizeof(uint16_t));
    carved("hidden gradient parts", a.part, (size_t)p.n_split * p.Rp * a.D * sizeof(float));
  }
  return hipSuccess;
}
hipError_t launch_head_zero(uint16_t*, int64_t, int, int, hipStream_t) {
  ++hoststub::g_launches;
  return hipSuccess;
}

}  // namespace specv

namespace {

int g_fail = 0;
#define CHECK(cond, ...)                                  \
  do {                                                    \
    if (!(cond)) {                                        \
      fprintf(stderr, "FAIL line %d: ", __LINE__);        \
      fprintf(stderr, __VA_ARGS__);                       \
      fprintf(stderr, "\n");                              \
      ++g_fail;                                           \
    }                                                     \
  } while (0)

void* const kDev = (void*)0x100000;
void* const kDev2 = (void*)0x200000;
void* const kDev3 = (void*)0x300000;

struct HostWs {
  void* p = nullptr;
  size_t n = 0;
  explicit HostWs(size_t bytes) : n(bytes) {
    if (bytes && posix_memalign(&p, 256, bytes) != 0) p = nullptr;
    hoststub::g_ws = {p, bytes};
  }
  ~HostWs() { free(p); }
};

void topk(int R, int V, int K) {
  HostWs ws(spec_row_topk_workspace_bytes(R, V, K));
  const int before = hoststub::g_launches;
  int rc = spec_row_topk(R, V, K, SPEC_BF16, kDev, V, 1.f, (int32_t*)kDev, (float*)kDev, nullptr, ws.p, ws.n, nullptr);
  CHECK(rc == SPEC_OK && hoststub::g_launches > before, "topk %d %d %d: rc %d", R, V, K, rc);
  CHECK(hoststub::check_disjoint() == 0, "topk: overlap");
  const int mid = hoststub::g_launches;
  rc = spec_row_topk(R, V, K, SPEC_BF16, kDev, V, 1.f, (int32_t*)kDev, (float*)kDev, nullptr, ws.p, ws.n - 1, nullptr);
  CHECK(rc == SPEC_ERR_WORKSPACE && hoststub::g_launches == mid, "topk: short workspace rc %d", rc);
}
void distill(int R, int V, int K, bool grad) {
  HostWs ws(spec_topk_distill_workspace_bytes(R, V, K, grad));
  int rc = spec_topk_distill(R, V, K, SPEC_F32, kDev, V, (int32_t*)kDev, (float*)kDev, nullptr, 1.f, nullptr, (float*)kDev,
                             nullptr, grad ? kDev2 : nullptr, V, ws.p, ws.n, nullptr);
  CHECK(rc == SPEC_OK, "distill %d %d %d: rc %d", R, V, K, rc);
  CHECK(hoststub::check_disjoint() == 0, "distill: overlap");
  rc = spec_topk_distill(R, V, K, SPEC_F32, kDev, V, (int32_t*)kDev, (float*)kDev, nullptr, 1.f, nullptr, (float*)kDev, nullptr,
                         grad ? kDev2 : nullptr, V, ws.p, ws.n - 1, nullptr);
  CHECK(rc == SPEC_ERR_WORKSPACE, "distill: short workspace rc %d", rc);
}
void head(int R, int V, int D, bool dh, bool dw) {
  HostWs ws(spec_lm_head_loss_workspace_bytes(R, V, D, dh || dw));
  int rc = spec_lm_head_loss(R, V, D, kDev, D, kDev, D, (int32_t*)kDev, 1.f, nullptr, (float*)kDev, nullptr, dh ? kDev2 : nullptr,
                             D, dw ? kDev3 : nullptr, D, ws.p, ws.n, nullptr);
  CHECK(rc == SPEC_OK, "head %d %d %d: rc %d", R, V, D, rc);
  CHECK(hoststub::check_disjoint() == 0, "head: overlap");
  rc = spec_lm_head_loss(R, V, D, kDev, D, kDev, D, (int32_t*)kDev, 1.f, nullptr, (float*)kDev, nullptr, dh ? kDev2 : nullptr, D,
                         dw ? kDev3 : nullptr, D, ws.p, ws.n - 1, nullptr);
  CHECK(rc == SPEC_ERR_WORKSPACE, "head: short workspace rc %d", rc);
}

}  // namespace

int main() {
  for (int R : {1, 7, 512})
    for (int V : {1, 8192, 8193, 151936})
      for (int K : {1, 64, 129, 256}) {
        topk(R, V, K);
        distill(R, V, K, true);
        distill(R, V, K, false);
      }
  for (int R : {1, 63, 64, 65, 128, 129, 448, 2100})
    for (int V : {1, 255, 32003, 151936})
      for (int D : {8, 264, 1032}) {
        head(R, V, D, true, true);
        head(R, V, D, true, false);
        head(R, V, D, false, true);
        head(R, V, D, false, false);
      }
  const int before = hoststub::g_launches;
  int32_t* const ip = (int32_t*)kDev;
  float* const fp = (float*)kDev;
  HostWs ws(1 << 20);
  auto tk = [&](int R, int V, int K, int type, const void* l, int64_t ld, float T, int32_t* oi, float* ol, void* w) {
    return spec_row_topk(R, V, K, type ? SPEC_BF16 : SPEC_F32, l, ld, T, oi, ol, nullptr, w, 1 << 20, nullptr);
  };
  CHECK(tk(0, 10, 2, 1, nullptr, 10, 1.f, ip, fp, ws.p) == SPEC_OK, "no rows");
  CHECK(tk(-1, 10, 2, 1, kDev, 10, 1.f, ip, fp, ws.p) == SPEC_ERR_INVALID, "R");
  CHECK(tk(2, 0, 2, 1, kDev, 10, 1.f, ip, fp, ws.p) == SPEC_ERR_INVALID, "V");
  CHECK(tk(2, 10, 0, 1, kDev, 10, 1.f, ip, fp, ws.p) == SPEC_ERR_INVALID, "K");
  CHECK(tk(2, 10, 257, 1, kDev, 10, 1.f, ip, fp, ws.p) == SPEC_ERR_UNSUPPORTED, "K large");
  CHECK(tk(2, (1 << 21) + 1, 2, 1, kDev, 1 << 22, 1.f, ip, fp, ws.p) == SPEC_ERR_UNSUPPORTED, "V large");
  CHECK(tk((1 << 22) + 1, 10, 2, 1, kDev, 10, 1.f, ip, fp, ws.p) == SPEC_ERR_UNSUPPORTED, "R large");
  CHECK(tk(1 << 22, 1 << 21, 2, 1, kDev, 1 << 21, 1.f, ip, fp, ws.p) == SPEC_ERR_WORKSPACE, "the largest call's size");
  CHECK(tk(2, 10, 2, 1, nullptr, 10, 1.f, ip, fp, ws.p) == SPEC_ERR_INVALID, "logits");
  CHECK(tk(2, 10, 2, 1, kDev, 9, 1.f, ip, fp, ws.p) == SPEC_ERR_INVALID, "ld");
  CHECK(tk(2, 10, 2, 1, kDev, 10, 1.f, nullptr, fp, ws.p) == SPEC_ERR_INVALID, "index");
  CHECK(tk(2, 10, 2, 1, kDev, 10, 1.f, ip, nullptr, ws.p) == SPEC_ERR_INVALID, "logit");
  CHECK(tk(2, 10, 2, 1, kDev, 10, 1.f, ip, fp, nullptr) == SPEC_ERR_WORKSPACE, "no workspace");
  CHECK(tk(2, 10, 2, 1, kDev, 10, 1.f, ip, fp, (char*)ws.p + 16) == SPEC_ERR_INVALID, "workspace alignment");
  for (float T : {0.f, -1.f, NAN, INFINITY, 1e-45f}) CHECK(tk(2, 10, 2, 1, kDev, 10, T, ip, fp, ws.p) == SPEC_ERR_INVALID, "T");

  auto td = [&](int R, int V, int K, const void* l, int64_t ld, const int32_t* x, const float* t, float T, float* lo, void* d,
                int64_t dld) {
    return spec_topk_distill(R, V, K, SPEC_BF16, l, ld, x, t, nullptr, T, nullptr, lo, nullptr, d, dld, ws.p, ws.n, nullptr);
  };
  CHECK(td(0, 10, 2, nullptr, 10, nullptr, nullptr, 1.f, nullptr, nullptr, 0) == SPEC_OK, "no rows");
  CHECK(td(2, 10, 2, nullptr, 10, ip, fp, 1.f, fp, nullptr, 0) == SPEC_ERR_INVALID, "logits");
  CHECK(td(2, 10, 2, kDev, 10, nullptr, fp, 1.f, fp, nullptr, 0) == SPEC_ERR_INVALID, "index");
  CHECK(td(2, 10, 2, kDev, 10, ip, nullptr, 1.f, fp, nullptr, 0) == SPEC_ERR_INVALID, "teacher");
  CHECK(td(2, 10, 2, kDev, 10, ip, fp, 1.f, nullptr, nullptr, 0) == SPEC_ERR_INVALID, "loss");
  CHECK(td(2, 10, 2, kDev, 9, ip, fp, 1.f, fp, nullptr, 0) == SPEC_ERR_INVALID, "ld");
  CHECK(td(2, 10, 2, kDev, 10, ip, fp, 1.f, fp, kDev2, 9) == SPEC_ERR_INVALID, "d_ld");
  CHECK(td(2, 10, 2, kDev, 10, ip, fp, 1.f, fp, kDev, 11) == SPEC_ERR_INVALID, "in place with another stride");
  CHECK(td(2, 10, 257, kDev, 10, ip, fp, 1.f, fp, nullptr, 0) == SPEC_ERR_UNSUPPORTED, "K large");
  CHECK(td(2, 10, 2, kDev, 10, ip, fp, 0.f, fp, nullptr, 0) == SPEC_ERR_INVALID, "T");

  auto hl = [&](int R, int V, int D, const void* h, int64_t hld, const void* w, int64_t wld, const int32_t* y, float T, float* lo,
                void* dh, int64_t dhld, void* dw, int64_t dwld) {
    return spec_lm_head_loss(R, V, D, h, hld, w, wld, y, T, nullptr, lo, nullptr, dh, dhld, dw, dwld, ws.p, ws.n, nullptr);
  };
  CHECK(hl(0, 10, 64, nullptr, 64, nullptr, 64, nullptr, 1.f, nullptr, nullptr, 0, nullptr, 0) == SPEC_OK, "no rows");
  CHECK(hl(0, 10, 64, nullptr, 64, nullptr, 64, nullptr, 1.f, nullptr, nullptr, 0, kDev, 32) == SPEC_ERR_INVALID, "no rows, dw_ld");
  CHECK(hl(-1, 10, 64, kDev, 64, kDev, 64, ip, 1.f, fp, nullptr, 0, nullptr, 0) == SPEC_ERR_INVALID, "R");
  CHECK(hl(2, 10, 64, nullptr, 64, kDev, 64, ip, 1.f, fp, nullptr, 0, nullptr, 0) == SPEC_ERR_INVALID, "hidden");
  CHECK(hl(2, 10, 64, kDev, 64, kDev, 64, nullptr, 1.f, fp, nullptr, 0, nullptr, 0) == SPEC_ERR_INVALID, "targets");
  CHECK(hl(2, 10, 64, kDev, 64, kDev, 64, ip, 1.f, nullptr, nullptr, 0, nullptr, 0) == SPEC_ERR_INVALID, "loss");
  CHECK(hl(2, 10, 64, kDev, 56, kDev, 64, ip, 1.f, fp, nullptr, 0, nullptr, 0) == SPEC_ERR_INVALID, "h_ld");
  CHECK(hl(2, 10, 64, kDev, 64, kDev, 64, ip, 1.f, fp, kDev2, 56, nullptr, 0) == SPEC_ERR_INVALID, "dh_ld");
  CHECK(hl(2, 10, 60, kDev, 64, kDev, 64, ip, 1.f, fp, nullptr, 0, nullptr, 0) == SPEC_ERR_UNSUPPORTED, "D");
  CHECK(hl(2, 10, 64, kDev, 68, kDev, 64, ip, 1.f, fp, nullptr, 0, nullptr, 0) == SPEC_ERR_UNSUPPORTED, "h_ld off the grid");
  CHECK(hl(2, 10, 64, (char*)kDev + 8, 64, kDev, 64, ip, 1.f, fp, nullptr, 0, nullptr, 0) == SPEC_ERR_UNSUPPORTED, "base");
  CHECK(hl(2, 10, 64, kDev, 64, kDev, 64, ip, 1.f, fp, (char*)kDev2 + 8, 64, nullptr, 0) == SPEC_ERR_UNSUPPORTED, "d_hidden base");
  CHECK(hl(2, 10, 64, kDev, 64, kDev2, 64, ip, 1.f, fp, kDev, 64, nullptr, 0) == SPEC_ERR_INVALID, "d_hidden over hidden");
  CHECK(hl(2, 10, 64, kDev, 64, kDev2, 64, ip, 1.f, fp, nullptr, 0, kDev2, 64) == SPEC_ERR_INVALID, "d_weight over weight");
  CHECK(hl(2, 10, 64, kDev, (int64_t)1 << 22, kDev, 64, ip, 1.f, fp, nullptr, 0, nullptr, 0) == SPEC_ERR_UNSUPPORTED, "h_ld large");
  CHECK(hl(2, 10, 64, kDev, 64, kDev, 64, ip, 0.f, fp, nullptr, 0, nullptr, 0) == SPEC_ERR_INVALID, "T");
  CHECK(hl(1 << 22, 1 << 21, 1 << 21, kDev, 1 << 21, kDev, 1 << 21, ip, 1.f, fp, kDev2, 1 << 21, kDev3, 1 << 21) != SPEC_OK,
        "the largest sizes");
  CHECK(hoststub::g_launches == before, "a refused call launched");
  printf("%d launches, %d failures\n", hoststub::g_launches, g_fail + hoststub::g_errors);
  return g_fail + hoststub::g_errors ? 1 : 0;
}
