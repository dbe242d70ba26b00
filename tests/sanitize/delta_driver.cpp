// delta_driver.cpp -- runs the host-side code of include/pararnn_delta.h that
// needs no GPU, for a build with AddressSanitizer and
// UndefinedBehaviorSanitizer: sizes of workspaces and saved states over a sweep
// of shapes (tiny, ragged, at the limits, invalid), and argument checks of every
// entry point, each called so that it returns before its first HIP call.
// Exit status 0 when every status is the documented one.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "../../include/pararnn_delta.h"

static int failures = 0;
#define CHECK(cond, ...)                     \
  do {                                       \
    if (!(cond)) {                           \
      fprintf(stderr, "FAIL: " __VA_ARGS__); \
      fprintf(stderr, "\n");                 \
      ++failures;                            \
    }                                        \
  } while (0)

// never dereferenced: every call below returns before it touches memory
template <class T = void>
static T* fake(uintptr_t k) { return reinterpret_cast<T*>(k * 4096); }

struct Views {
  pararnn_view q, k, v, g;
};

static int scan(const Views& x, void* ws, size_t n, const pararnn_delta_opts& o, void* saved = nullptr) {
  return pararnn_delta_scan(&x.q, &x.k, &x.v, &x.g, fake<float>(5), nullptr, fake(6), nullptr, saved, ws, n, &o, nullptr);
}
static int adjoint(const Views& x, const Views& d, void* ws, size_t n, const pararnn_delta_opts& o) {
  return pararnn_delta_scan_adjoint(&x.q, &x.k, &x.v, &x.g, fake<float>(5), fake(7), fake(8), nullptr, &d.q, &d.k, &d.v,
                                    &d.g, nullptr, nullptr, ws, n, &o, nullptr);
}

static void delta(int B, int L, int H, int HV, int dk, int dv, int dtype) {
  pararnn_delta_opts o = {B, L, H, HV, dk, dv, dtype, 8.0f, 1e-6f, 1.0f, nullptr, nullptr};
  size_t n[3] = {1, 1, 1};
  const int rc[3] = {pararnn_delta_workspace_bytes(0, &o, &n[0]), pararnn_delta_workspace_bytes(1, &o, &n[1]),
                     pararnn_delta_saved_bytes(&o, &n[2])};
  CHECK(rc[0] == rc[1] && rc[0] == rc[2], "one answer for every size");
  if (B < 1 || L < 1 || H < 1 || HV < H || HV % H || dk < 1 || dk > 128 || dv < 1 || dv > 512)
    CHECK(rc[0] == PARARNN_EINVAL, "invalid sizes %d %d %d %d %d %d", B, L, H, HV, dk, dv);
  if (rc[0]) return;
  CHECK(dtype == 0 || dtype == 1, "type");
  for (size_t x : n) CHECK(x % 256 == 0 && x > 0, "whole lines");
  CHECK(n[1] > n[0], "the adjoint's is the larger");
  const int64_t nk = int64_t(H) * dk, nv = int64_t(HV) * dv, ng = 2 * int64_t(HV);
  if (nk > (1 << 22) || nv > (1 << 22) || ng > (1 << 22)) return;  // further apart than a view may be
  const Views x = {{fake(1), L * nk, nk}, {fake(2), L * nk, nk}, {fake(3), L * nv, nv}, {fake(4), L * ng, ng}};
  for (int masks = 0; masks < 4; ++masks) {  // too small by a byte, with every mask
    o.lengths = masks & 1 ? fake<const int32_t>(20) : nullptr;
    o.reset = masks & 2 ? fake<const uint8_t>(21) : nullptr;
    CHECK(scan(x, fake(9), n[0] - 1, o) == PARARNN_EWORKSPACE, "workspace %d %d %d", B, L, HV);
    CHECK(adjoint(x, x, fake(9), n[1] - 1, o) == PARARNN_EWORKSPACE, "workspace, adjoint %d %d %d", B, L, HV);
  }
  CHECK(scan(x, nullptr, n[0], o) == PARARNN_EINVAL, "no workspace");
  CHECK(scan(x, fake<char>(9) + 16, n[0], o) == PARARNN_EUNSUPPORTED, "workspace off its line");
  CHECK(scan(x, fake(9), n[0], o, fake<char>(9) + 16) == PARARNN_EUNSUPPORTED, "saved off its line");
  for (int i = 0; i < 4; ++i) {
    Views y = x;
    pararnn_view* const all[4] = {&y.q, &y.k, &y.v, &y.g};
    pararnn_view& z = *all[i];
    const pararnn_view was = z;
    z.p = nullptr;
    CHECK(scan(y, fake(9), n[0], o) == PARARNN_EINVAL && adjoint(x, y, fake(9), n[1], o) == PARARNN_EINVAL, "no tensor");
    z = was;
    z.token -= 1;
    CHECK(scan(y, fake(9), n[0], o) == PARARNN_EINVAL && adjoint(y, x, fake(9), n[1], o) == PARARNN_EINVAL, "tokens overlap");
    z.token = (1 << 22) + 1;
    CHECK(scan(y, fake(9), n[0], o) == PARARNN_EINVAL, "tokens too far apart");
    z = was;
    if (B > 1) {
      for (int64_t batch : {int64_t(-1), int64_t(0), was.batch - 1, INT64_MAX}) {
        z.batch = batch;
        CHECK(scan(y, fake(9), n[0], o) == PARARNN_EINVAL, "rows overlap, or too far apart");
      }
      z = was;
    }
    z.p = static_cast<const char*>(was.p) + 1;
    CHECK(scan(y, fake(9), n[0], o) == PARARNN_EUNSUPPORTED, "alignment");
  }
  for (float bad : {0.0f, -1.0f, INFINITY, NAN}) {
    o.c = bad;
    CHECK(scan(x, fake(9), n[0], o) == PARARNN_EINVAL, "c");
    o.c = 8.0f;
    o.eps = bad;
    CHECK(scan(x, fake(9), n[0], o) == PARARNN_EINVAL, "eps");
    o.eps = 1e-6f;
    o.scale = bad;
    if (!isfinite(bad)) CHECK(scan(x, fake(9), n[0], o) == PARARNN_EINVAL, "scale");
    o.scale = 1.0f;
  }
  for (int S : {-1, 0, B - 1})
    CHECK(pararnn_delta_step(&x.q, &x.k, &x.v, &x.g, fake<float>(5), nullptr, fake<float>(6), fake(7), S, &o, nullptr) ==
              PARARNN_EINVAL, "step pool");
  if (L > 1)
    CHECK(pararnn_delta_step(&x.q, &x.k, &x.v, &x.g, fake<float>(5), nullptr, fake<float>(6), fake(7), B, &o, nullptr) ==
              PARARNN_EINVAL, "a step of several tokens");
}

static void norm(int64_t N, int D, int group, int dtype, float eps, int64_t row) {
  pararnn_norm_block_opts o = {N, D, group, dtype, 0, eps, row, row, row};
  for (int residual : {0, 1}) {
    size_t n = 1;
    const int rc = pararnn_norm_block_workspace_bytes(&o, residual, &n);
    if (N < 1 || D < 1 || D > 16384 || group < 1 || group > D || D % group || !(eps >= 0.0f) || !isfinite(eps) || row < D)
      CHECK(rc == PARARNN_EINVAL, "invalid norm options %lld %d %d", static_cast<long long>(N), D, group);
    if (rc) continue;
    CHECK(n % 256 == 0 && n >= sizeof(float) * group, "a partial row at least");
    const void* s = residual ? fake(2) : nullptr;
    const float* w_next = residual ? fake<float>(4) : nullptr;
    const int got = pararnn_norm_block_adjoint(fake(1), nullptr, s, fake<float>(3), nullptr, w_next, fake(5), nullptr,
                                               fake(6), nullptr, residual ? fake(7) : nullptr, fake<float>(8), nullptr,
                                               nullptr, fake(9), 0, &o, nullptr);
    CHECK(got == PARARNN_EWORKSPACE || got == PARARNN_EUNSUPPORTED, "norm workspace");
    CHECK(pararnn_norm_block(nullptr, nullptr, nullptr, fake<float>(3), nullptr, nullptr, nullptr, fake(6), nullptr, &o,
                             nullptr) == PARARNN_EINVAL, "NULL x");
    CHECK(pararnn_norm_block(fake(1), nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, fake(6), nullptr, &o, nullptr) ==
              PARARNN_EINVAL, "neither w nor a residual");
    o.out = 1;
    CHECK(pararnn_norm_block(fake(1), nullptr, nullptr, fake<float>(3), nullptr, nullptr, nullptr, fake(6), nullptr, &o,
                             nullptr) == PARARNN_EINVAL, "8 bits without scales");
    o.out = 2;
    CHECK(pararnn_norm_block(fake(1), nullptr, nullptr, fake<float>(3), nullptr, nullptr, nullptr, fake(6), nullptr, &o,
                             nullptr) == PARARNN_EINVAL, "no such output");
    o.out = 0;
  }
}

int main() {
  const int lengths[] = {-1, 0, 1, 63, 64, 65, 1000, 65536, 2147480000, 2147483647};
  for (int B : {-1, 0, 1, 2, 65, 2147483647})
    for (int L : lengths)
      for (int H : {0, 1, 3, 2147483647})
        for (int HV : {0, 1, 3, 6, 2147483647})
          for (int dk : {0, 1, 64, 65, 128, 129})
            for (int dv : {0, 1, 64, 100, 512, 513})
              for (int dtype : {-1, 0, 1, 2}) delta(B, L, H, HV, dk, dv, dtype);
  size_t n = 0;
  const pararnn_delta_opts o = {1, 1, 1, 1, 8, 8, 0, 8.0f, 1e-6f, 1.0f, nullptr, nullptr};
  CHECK(pararnn_delta_workspace_bytes(0, nullptr, &n) == PARARNN_EINVAL, "NULL options");
  CHECK(pararnn_delta_workspace_bytes(2, &o, &n) == PARARNN_EINVAL, "neither pass");
  CHECK(pararnn_delta_workspace_bytes(0, &o, nullptr) == PARARNN_EINVAL, "NULL size");
  CHECK(pararnn_delta_saved_bytes(&o, nullptr) == PARARNN_EINVAL, "NULL size of saved");

  for (int64_t N : {int64_t(-1), int64_t(0), int64_t(1), int64_t(4999), int64_t(1) << 31, int64_t(1) << 62, INT64_MAX})
    for (int D : {-1, 0, 1, 96, 128, 1000, 4096, 8192, 16384, 16385, 2147483647})
      for (int group : {-1, 0, 1, 3, 32, 128, 1000, 2147483647})
        for (float eps : {0.0f, 1e-6f, -1.0f, NAN, INFINITY})
          for (int dtype : {0, 1, 2})
            for (int64_t row : {int64_t(D) - 1, int64_t(D), int64_t(1) << 40, INT64_MAX}) norm(N, D, group, dtype, eps, row);

  const int sizes[] = {-1, 0, 1, 16, 257, 4096, 131071, 131072, 2147480000, 2147483647};
  for (int M : sizes)
    for (int N : sizes)
      for (int K : sizes) {
        const pararnn_int8_opts i = {M, N, K, 1};
        const int rc = pararnn_matmul_int8(fake(1), fake<float>(2), fake(3), fake<float>(4), nullptr, fake<char>(5) + 1, &i,
                                           nullptr);
        if (M < 1 || N < 1 || K < 1 || K > 131071) CHECK(rc == PARARNN_EINVAL, "product sizes %d %d %d", M, N, K);
        else CHECK(rc == PARARNN_EUNSUPPORTED || rc == PARARNN_EINVAL, "y at an odd byte %d %d %d", M, N, K);
      }
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
