// host_common.h -- what the host sides of the layer operators share: sizes,
// alignment and the launch. Host code only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../../include/pararnn.h"

namespace pararnn {
namespace {

constexpr int kCUs = 256;
constexpr size_t kAlign = 256;
size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int check_hip(hipError_t e) { return e == hipSuccess ? PARARNN_OK : PARARNN_EHIP; }

// A launch's size in threads is a 32-bit number: a larger one would run as its
// low 32 bits (8388609 workgroups of 512 as one), without an error.
constexpr long long kMaxThreads = 4294967295LL;

template <typename F, typename... Args>
int launch(F kernel, long long grid, int block, hipStream_t s, Args... args) {
  if (grid > kMaxThreads / block) return PARARNN_EINVAL;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(block), 0, s, args...);
  return check_hip(hipGetLastError());
}

bool dtype_ok(int32_t d) { return d == PARARNN_F32 || d == PARARNN_BF16; }

}  // namespace
}  // namespace pararnn
