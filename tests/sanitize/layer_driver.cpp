// layer_driver.cpp -- runs the host-side code of include/pararnn_layer.h that
// needs no GPU, for a build with AddressSanitizer and
// UndefinedBehaviorSanitizer: workspace sizes over a sweep of shapes (tiny,
// ragged, at the limits, invalid), and argument checks of every entry point,
// each called so that it returns before its first HIP call.
// Exit status 0 when every status is the documented one.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "../../include/pararnn_layer.h"

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

static void gated(int B, int L, int D) {
  for (int dtype : {-1, 0, 1, 2})
    for (float c : {8.0f, 0.0f, -1.0f, INFINITY, NAN}) {
      const bool bad_c = !(c > 0.0f) || !isfinite(c);
      pararnn_gated_opts o = {B, L, D, dtype, c, nullptr, nullptr};
      size_t n[2] = {1, 1};
      int rc[2];
      for (int adj : {0, 1}) {
        rc[adj] = pararnn_gated_workspace_bytes(adj, &o, &n[adj]);
        if (bad_c || B < 1 || L < 1 || D < 1) CHECK(rc[adj] == PARARNN_EINVAL, "invalid sizes %d %d %d", B, L, D);
        else if (rc[adj] == PARARNN_OK) CHECK(n[adj] % 256 == 0, "whole lines");
      }
      if (rc[0] || rc[1]) continue;
      CHECK(dtype == 0 || dtype == 1, "type");
      // too small by one byte, with every mask: the size covers all of them
      for (int masks = 0; masks < 4; ++masks) {
        o.lengths = masks & 1 ? fake<const int32_t>(20) : nullptr;
        o.reset = masks & 2 ? fake<const uint8_t>(21) : nullptr;
        if (n[0])
          CHECK(pararnn_gated_scan(fake(1), fake<float>(2), nullptr, fake(3), nullptr, nullptr, fake(4), 0, &o,
                                   nullptr) == PARARNN_EWORKSPACE, "no workspace %d %d %d", B, L, D);
        if (n[1])
          CHECK(pararnn_gated_scan_adjoint(fake(1), fake<float>(2), fake<float>(3), fake(4), nullptr, fake(5), nullptr,
                                           nullptr, fake(6), 0, &o, nullptr) == PARARNN_EWORKSPACE,
                "no workspace, adjoint %d %d %d", B, L, D);
        // a bf16 pointer at an odd byte, an fp32 one off its four
        char* odd = fake<char>(1) + 1;
        CHECK(pararnn_gated_scan(odd, fake<float>(2), nullptr, fake(3), nullptr, nullptr, fake(4), n[0], &o, nullptr) ==
                  PARARNN_EUNSUPPORTED, "alignment");
      }
      CHECK(pararnn_gated_scan(nullptr, fake<float>(2), nullptr, fake(3), nullptr, nullptr, fake(4), n[0], &o,
                               nullptr) == PARARNN_EINVAL, "NULL u");
    }
}

static void norm(int64_t N, int D) {
  for (int dtype : {-1, 0, 1, 2})
    for (float eps : {0.0f, 1e-6f, -1.0f, NAN}) {
      pararnn_norm_opts o = {N, D, dtype, 0, eps};
      const size_t n = pararnn_norm_workspace_bytes(&o);
      const bool ok = N >= 1 && D >= 1 && D <= 16384 && eps >= 0.0f && dtype >= 0 && dtype <= 1;
      if (!ok) CHECK(n == 0, "invalid norm options");
      else if (n) CHECK(n % 256 == 0 && n >= sizeof(float) * D, "a partial row at least");
      if (n)
        CHECK(pararnn_norm_residual_adjoint(fake(1), fake<float>(2), fake(3), nullptr, fake(4), fake<float>(5), fake(6),
                                            n - 1, &o, nullptr) == PARARNN_EWORKSPACE, "norm workspace");
      CHECK(pararnn_norm_residual(nullptr, nullptr, fake<float>(2), nullptr, fake(3), nullptr, &o, nullptr) ==
                PARARNN_EINVAL, "NULL x");
      o.out = 1;
      CHECK(pararnn_norm_residual(fake(1), nullptr, fake<float>(2), nullptr, fake(3), nullptr, &o, nullptr) ==
                PARARNN_EINVAL, "8 bits without scales");
    }
}

int main() {
  const int sizes[] = {-1, 0, 1, 2, 63, 64, 65, 96, 97, 257, 1000, 4097, 65536, 2147480000, 2147483647};
  for (int B : sizes)
    for (int L : sizes)
      for (int D : sizes) gated(B, L, D);
  for (int64_t N : {int64_t(-1), int64_t(0), int64_t(1), int64_t(4999), int64_t(1) << 31, int64_t(1) << 62, INT64_MAX})
    for (int D : sizes) norm(N, D);
  for (int L : sizes) {
    const int r = pararnn_gated_saved_rows(L);
    CHECK(L < 1 ? r == 0 : static_cast<int64_t>(r) * 96 >= L && static_cast<int64_t>(r - 1) * 96 < L, "saved rows");
  }
  CHECK(pararnn_gated_workspace_bytes(0, nullptr, nullptr) == PARARNN_EINVAL, "NULL options");
  CHECK(pararnn_norm_workspace_bytes(nullptr) == 0, "NULL norm options");

  for (int B : {-1, 0, 1, 2147483647})
    for (int S : {-1, 0, 1})
      if (B != 1 || S != 1)
        CHECK(pararnn_gated_step(fake(1), fake<float>(2), nullptr, fake<float>(3), fake(4), B, 64, S, 0, 8.0f,
                                 nullptr) == PARARNN_EINVAL, "step sizes");
  CHECK(pararnn_gated_step(fake(1), fake<float>(2), nullptr, fake<float>(3), fake(4), 1, 64, 1, 2, 8.0f, nullptr) ==
            PARARNN_EUNSUPPORTED, "step type");

  for (int M : sizes)
    for (int N : sizes)
      for (int K : sizes)
        for (int rows : {0, 1, 128}) {
          pararnn_matmul_opts o = {M, N, K, rows, 0, 1};
          if (rows == 0 || M < 1 || N < 1 || K < 1 || M > 2147483647 - 256 || N > 2147483647 - 256 || K > (1 << 22) ||
              (M > 2000000000 && N > 2000000000))
            CHECK(pararnn_matmul_fp8(fake(1), fake(2), fake(3), fake(4), nullptr, fake(5), &o, nullptr) ==
                      PARARNN_EINVAL, "product sizes %d %d %d", M, N, K);
          else
            CHECK(pararnn_matmul_fp8(fake(1), fake(2), fake(3), fake(4), fake<float>(6), fake<char>(5) + 1, &o,
                                     nullptr) == PARARNN_EUNSUPPORTED, "y at an odd byte");
        }
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
