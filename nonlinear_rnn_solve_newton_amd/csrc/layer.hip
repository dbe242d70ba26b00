// layer.hip -- host side of the C ABI declared in include/pararnn_layer.h:
// argument checks, the choice of a launch shape, workspace carving and the
// launches, all asynchronous on the caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>

#include "../../include/pararnn_layer.h"
#include "gated_scan.h"

namespace pararnn {
namespace {

constexpr size_t kAlign = 256;
size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int check_hip(hipError_t e) { return e == hipSuccess ? PARARNN_OK : PARARNN_EHIP; }

template <typename F, typename... Args>
int launch(F kernel, long long grid, int block, hipStream_t s, Args... args) {
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(block), 0, s, args...);
  return check_hip(hipGetLastError());
}

// clears n16 16-byte words (a kernel rather than a memset: graphs of the
// caller's stream capture it)
__global__ void __launch_bounds__(256) clear_kernel(f32x4* p, long long n16) {
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n16; i += 256LL * gridDim.x)
    p[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}
int clear(void* p, size_t bytes, hipStream_t s) {
  const long long n16 = static_cast<long long>(bytes / 16);
  long long blocks = ceil_div(n16, 256);
  if (blocks > 4096) blocks = 4096;
  return launch(clear_kernel, blocks, 256, s, static_cast<f32x4*>(p), n16);
}

// widest group of channels in {4, 2, 1}, at most cmax, that divides D and that
// every pointer is aligned for: es bytes per element for `typed`, 4 for `f32`
int pick_c(int cmax, int D, size_t es, std::initializer_list<const void*> typed,
           std::initializer_list<const void*> f32) {
  for (int C : {4, 2, 1}) {
    if (C > cmax || D % C) continue;
    bool ok = true;
    for (const void* q : typed) ok = ok && (!q || aligned(q, es * C));
    for (const void* q : f32) ok = ok && (!q || aligned(q, sizeof(float) * C));
    if (ok) return C;
  }
  return 0;
}

// ---------------------------------------------------------------------------
// gated scan

// Launch shapes: C channels per lane, T steps per lane, LL lane groups; 8 waves
template <class UT, int C> struct ScanShape;
template <> struct ScanShape<bf16, 4> { static constexpr int T = 8, LL = 4; };
template <> struct ScanShape<bf16, 2> { static constexpr int T = 16, LL = 2; };
template <> struct ScanShape<bf16, 1> { static constexpr int T = 32, LL = 1; };
template <> struct ScanShape<float, 2> { static constexpr int T = 8, LL = 4; };
template <> struct ScanShape<float, 1> { static constexpr int T = 16, LL = 2; };
template <int C> struct AdjShape;
template <> struct AdjShape<2> { static constexpr int T = 8, LL = 2; };
template <> struct AdjShape<1> { static constexpr int T = 16, LL = 1; };
constexpr int kWaves = 8;
constexpr int kScanChunk = 256;
static_assert(kWaves * AdjShape<2>::T * AdjShape<2>::LL == kGatedSave &&
              kWaves * AdjShape<1>::T * AdjShape<1>::LL == kGatedSave, "adjoint chunk");

int scan_cw(int dtype, int C, bool adj) {
  if (adj) return C == 2 ? 64 / AdjShape<2>::LL * 2 : 64 / AdjShape<1>::LL;
  if (dtype == PARARNN_BF16)
    return C == 4 ? 64 / ScanShape<bf16, 4>::LL * 4 : C == 2 ? 64 / ScanShape<bf16, 2>::LL * 2 : 64;
  return C == 2 ? 64 / ScanShape<float, 2>::LL * 2 : 64 / ScanShape<float, 1>::LL;
}
int scan_cmax(int dtype, bool adj) { return adj ? 2 : dtype == PARARNN_BF16 ? 4 : 2; }

struct GatedLayout {
  size_t ctr = 0, carry = 0, agg = 0, clear_end = 0, part = 0, total = 0;
  int nchunks = 0, ntiles_d = 0, group = 1;
};

GatedLayout gated_layout(const pararnn_gated_opts* o, bool adj, int C) {
  GatedLayout y;
  const int chunk = adj ? kGatedSave : kScanChunk, cw = scan_cw(o->dtype, C, adj);
  y.nchunks = static_cast<int>(ceil_div(o->L, chunk));
  y.ntiles_d = static_cast<int>(ceil_div(o->D, cw));
  const size_t slots = static_cast<size_t>(o->B) * y.ntiles_d * cw;
  y.group = 8;
  size_t off = 0;
  if (y.nchunks > 1) {
    off = round_up(sizeof(uint32_t));
    y.carry = off;
    off = round_up(off + sizeof(uint64_t) * slots * (ceil_div(y.nchunks, y.group) + 1));
    y.agg = off;
    if (y.group > 1) off = round_up(off + sizeof(uint64_t) * slots * 2 * y.nchunks);
  }
  y.clear_end = off;
  y.part = off;
  if (adj) off = round_up(off + sizeof(float) * y.nchunks * static_cast<size_t>(o->B) * o->D);
  y.total = off > kAlign ? off : kAlign;
  return y;
}

bool gated_ok(const pararnn_gated_opts* o, bool adj) {
  if (!o || o->B < 1 || o->L < 1 || o->D < 1) return false;
  if (!(o->c > 0.0f) || !isfinite(o->c)) return false;
  if (o->L > 2147483647 - 2 * kScanChunk) return false;  // step numbers of a last partial chunk
  if (static_cast<double>(o->B) * o->L * o->D * 12 > 9.0e18) return false;
  for (int C = 1; C <= scan_cmax(o->dtype, adj); C *= 2) {
    const double wgs = static_cast<double>(o->B) * ceil_div(o->D, scan_cw(o->dtype, C, adj)) *
                       ceil_div(o->L, adj ? kGatedSave : kScanChunk);
    if (wgs > 2.0e9) return false;
  }
  // one chunk is addressed with 32-bit offsets below 2^31
  return static_cast<double>(kScanChunk) * 3 * o->D * 4 < 2147483648.0;
}
bool dtype_ok(int dtype) { return dtype == PARARNN_F32 || dtype == PARARNN_BF16; }

template <class UT, int C, bool RST>
int launch_gated(const GatedArgs& a, bool adj, hipStream_t s) {
  const long long grid = static_cast<long long>(a.B) * a.ntiles_d * a.nchunks;
  const GatedArgs& b = a;
  if (adj) {
    if constexpr (C <= 2) {
      using K = AdjShape<C>;
      return launch(gated_adjoint_kernel<UT, C, K::T, kWaves, K::LL, 2, RST>, grid, 64 * kWaves, s, b);
    }
    return PARARNN_EUNSUPPORTED;
  }
  if constexpr (C == 4 && sizeof(UT) == 4) return PARARNN_EUNSUPPORTED;
  else {
    using K = ScanShape<UT, C>;
    static_assert(K::T * K::LL * kWaves == kScanChunk, "chunk");
    return launch(gated_scan_kernel<UT, C, K::T, kWaves, K::LL, 4, RST>, grid, 64 * kWaves, s, b);
  }
}
template <class UT>
int launch_gated_c(int C, const GatedArgs& a, bool adj, hipStream_t s) {
  const bool r = a.reset != nullptr;
  if (C == 4) return r ? launch_gated<UT, 4, true>(a, adj, s) : launch_gated<UT, 4, false>(a, adj, s);
  if (C == 2) return r ? launch_gated<UT, 2, true>(a, adj, s) : launch_gated<UT, 2, false>(a, adj, s);
  return r ? launch_gated<UT, 1, true>(a, adj, s) : launch_gated<UT, 1, false>(a, adj, s);
}

int gated(bool adj, GatedArgs& a, float* dlam, void* ws, size_t ws_bytes, const pararnn_gated_opts* o, int C,
          hipStream_t stream) {
  const GatedLayout y = gated_layout(o, adj, C);
  if (ws_bytes < y.total) return PARARNN_EWORKSPACE;
  if (!aligned(ws, kAlign)) return PARARNN_EUNSUPPORTED;
  char* w = static_cast<char*>(ws);
  a.lengths = o->lengths;
  a.reset = o->reset;
  a.carry = reinterpret_cast<unsigned long long*>(w + y.carry);
  a.agg = reinterpret_cast<unsigned long long*>(w + y.agg);
  a.ctr = reinterpret_cast<unsigned int*>(w + y.ctr);
  if (dlam) a.dl_part = reinterpret_cast<float*>(w + y.part);
  a.B = o->B;
  a.L = o->L;
  a.D = o->D;
  a.nchunks = y.nchunks;
  a.ntiles_d = y.ntiles_d;
  a.group = y.group;
  a.c = o->c;
  if (y.clear_end) {
    const int rc = clear(w, y.clear_end, stream);
    if (rc) return rc;
  }
  const int rc = o->dtype == PARARNN_BF16 ? launch_gated_c<bf16>(C, a, adj, stream)
                                          : launch_gated_c<float>(C, a, adj, stream);
  if (rc || !dlam) return rc;
  return launch(column_sum_kernel, ceil_div(o->D, kSumCols), kSumCols * kSumGroups, stream,
                static_cast<const float*>(a.dl_part), dlam, static_cast<long long>(y.nchunks) * o->B,
                static_cast<int>(o->D), a.lam, o->c);
}

}  // namespace
}  // namespace pararnn

using namespace pararnn;

extern "C" size_t pararnn_gated_workspace_bytes(int32_t adjoint, const pararnn_gated_opts* o) {
  if ((adjoint != 0 && adjoint != 1) || !gated_ok(o, adjoint != 0) || !dtype_ok(o->dtype)) return 0;
  size_t n = 0;
  for (int C = 1; C <= scan_cmax(o->dtype, adjoint != 0); C *= 2) {
    const size_t t = gated_layout(o, adjoint != 0, C).total;
    n = t > n ? t : n;
  }
  return n;
}

extern "C" int32_t pararnn_gated_saved_rows(int32_t L) {
  return L < 1 ? 0 : static_cast<int32_t>(ceil_div(L, kGatedSave));
}

extern "C" int32_t pararnn_gated_scan(const void* u, const float* lam, const float* h0, void* h, float* hT,
                                      float* saved, void* ws, size_t ws_bytes, const pararnn_gated_opts* o,
                                      void* stream) {
  if (!gated_ok(o, false) || !u || !lam || !h || !ws) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = o->dtype == PARARNN_BF16 ? 2 : 4;
  const int C = pick_c(scan_cmax(o->dtype, false), o->D, es, {u, h}, {hT, saved});
  if (!C || !aligned(lam, 4) || !aligned(h0, 4) || !aligned(o->lengths, 4)) return PARARNN_EUNSUPPORTED;
  GatedArgs a;
  memset(&a, 0, sizeof(a));
  a.u = u;
  a.lam = lam;
  a.h0 = h0;
  a.h = h;
  a.hT = hT;
  a.saved = saved;
  return gated(false, a, nullptr, ws, ws_bytes, o, C, static_cast<hipStream_t>(stream));
}

extern "C" int32_t pararnn_gated_scan_adjoint(const void* u, const float* lam, const float* saved, const void* dh,
                                              const float* dhT, void* du, float* dlam, float* dh0, void* ws,
                                              size_t ws_bytes, const pararnn_gated_opts* o, void* stream) {
  if (!gated_ok(o, true) || !u || !lam || !saved || !dh || !du || !ws) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = o->dtype == PARARNN_BF16 ? 2 : 4;
  const int C = pick_c(scan_cmax(o->dtype, true), o->D, es, {u, dh, du}, {saved, dh0});
  if (!C || !aligned(lam, 4) || !aligned(dhT, 4) || !aligned(dlam, 4) || !aligned(o->lengths, 4))
    return PARARNN_EUNSUPPORTED;
  GatedArgs a;
  memset(&a, 0, sizeof(a));
  a.u = u;
  a.lam = lam;
  a.saved = const_cast<float*>(saved);
  a.dh = dh;
  a.dhT = dhT;
  a.du = du;
  a.dh0 = dh0;
  return gated(true, a, dlam, ws, ws_bytes, o, C, static_cast<hipStream_t>(stream));
}

extern "C" int32_t pararnn_gated_step(const void* u, const float* lam, const int32_t* slots, float* state, void* h,
                                      int32_t B, int32_t D, int32_t S, int32_t dtype, float c, void* stream_) {
  if (B < 1 || D < 1 || S < 1 || (!slots && S < B) || !u || !lam || !state || !h) return PARARNN_EINVAL;
  if (!(c > 0.0f) || !isfinite(c)) return PARARNN_EINVAL;
  if (!dtype_ok(dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = dtype == PARARNN_BF16 ? 2 : 4;
  const int C = pick_c(4, D, es, {u, h}, {lam, state});
  if (!C || !aligned(slots, 4)) return PARARNN_EUNSUPPORTED;
  const long long blocks = ceil_div(static_cast<long long>(B) * (D / C), 256);
  if (blocks > 2000000000LL) return PARARNN_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream_);
  auto go = [&](auto kernel, auto* up, auto* hp) { return launch(kernel, blocks, 256, s, up, lam, slots, state, hp, B, D, S, c); };
  if (dtype == PARARNN_BF16) {
    const bf16* up = static_cast<const bf16*>(u);
    bf16* hp = static_cast<bf16*>(h);
    return C == 4 ? go(gated_step_kernel<bf16, 4>, up, hp) : C == 2 ? go(gated_step_kernel<bf16, 2>, up, hp)
                                                                    : go(gated_step_kernel<bf16, 1>, up, hp);
  }
  const float* up = static_cast<const float*>(u);
  float* hp = static_cast<float*>(h);
  return C == 4 ? go(gated_step_kernel<float, 4>, up, hp) : C == 2 ? go(gated_step_kernel<float, 2>, up, hp)
                                                                   : go(gated_step_kernel<float, 1>, up, hp);
}
