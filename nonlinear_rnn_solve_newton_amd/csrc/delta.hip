// delta.hip -- host side of the C ABI declared in include/pararnn_delta.h:
// argument checks, the choice of a launch shape, workspace carving and the
// launches, all asynchronous on the caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <type_traits>
#include <utility>

#include "../../include/pararnn_delta.h"
#include "delta/delta_rule.h"
#include "layer/host_common.h"

namespace pararnn {
namespace {

// ---------------------------------------------------------------------------
// delta rule

constexpr int kMaxDk = 128, kMaxDv = 512;

bool delta_ok(const pararnn_delta_opts* o) {
  return o && o->B >= 1 && o->L >= 1 && o->H >= 1 && o->HV >= o->H && o->HV % o->H == 0 && o->dk >= 1 &&
         o->dk <= kMaxDk && o->dv >= 1 && o->dv <= kMaxDv && o->c > 0.0f && isfinite(o->c) && o->eps > 0.0f &&
         isfinite(o->eps) && isfinite(o->scale) && o->L <= 2147483647 - kDeltaChunk &&
         static_cast<long long>(o->B) * o->HV <= 2147483647LL &&
         static_cast<long long>(o->B) * o->HV * ceil_div(o->L, kDeltaChunk) <= kMaxThreads / 512;
}

// sizes of a call's pieces, in bytes (chunks of all value heads)
struct DeltaSizes {
  size_t frags, rows, states, ys, part;
};
DeltaSizes delta_sizes(const pararnn_delta_opts* o, bool adj) {
  const size_t chunks = static_cast<size_t>(o->B) * o->HV * ceil_div(o->L, kDeltaChunk);
  const size_t frag = o->dtype == PARARNN_BF16
                          ? (adj ? DeltaFrags<bf16, true>::ALL : DeltaFrags<bf16, false>::ALL)
                          : (adj ? DeltaFrags<float, true>::ALL : DeltaFrags<float, false>::ALL);
  return {round_up(chunks * frag * sizeof(bf16x8)), round_up(chunks * kRows * 64 * sizeof(float)),
          chunks * delta_tiles(o->dv) * delta_tiles(o->dk) * 1024, chunks * delta_tiles(o->dv) * 4096,
          round_up(chunks * sizeof(float))};
}

// every row and head starts at a multiple of `bytes`
bool rows_aligned(const pararnn_view* v, size_t es, int d, size_t bytes, int B) {
  return aligned(v->p, bytes) && d * es % bytes == 0 && v->token * es % bytes == 0 && (B == 1 || v->batch * es % bytes == 0);
}

constexpr long long kMaxToken = 1 << 22;  // 64 rows within 32-bit offsets
bool view_ok(const pararnn_view* v, const pararnn_delta_opts* o, long long packed) {
  if (!v || !v->p || v->token < packed || v->token > kMaxToken || v->batch > (1LL << 50)) return false;
  return o->B == 1 || v->batch >= static_cast<long long>(o->L - 1) * v->token + packed;
}
bool views_ok(const pararnn_view* q, const pararnn_view* k, const pararnn_view* v, const pararnn_view* g,
              const pararnn_delta_opts* o) {
  const long long nk = static_cast<long long>(o->H) * o->dk, nv = static_cast<long long>(o->HV) * o->dv;
  return view_ok(q, o, nk) && view_ok(k, o, nk) && view_ok(v, o, nv) && view_ok(g, o, 2LL * o->HV);
}
DeltaView view(const pararnn_view* v) { return {v->p, v->batch, v->token}; }

void delta_fill(DeltaArgs& a, const pararnn_view* q, const pararnn_view* k, const pararnn_view* v,
                const pararnn_view* gates, const float* lam, const pararnn_delta_opts* o, size_t es) {
  memset(&a, 0, sizeof(a));
  a.q = view(q);
  a.k = view(k);
  a.v = view(v);
  a.gates = view(gates);
  a.lam = lam;
  a.lengths = o->lengths;
  a.reset = o->reset;
  a.B = o->B;
  a.L = o->L;
  a.H = o->H;
  a.HV = o->HV;
  a.dk = o->dk;
  a.dv = o->dv;
  a.nc = static_cast<int>(ceil_div(o->L, kDeltaChunk));
  a.c = o->c;
  a.eps = o->eps;
  a.scale = o->scale;
}

template <class UT, bool EVEN, int DK, bool ADJ>
int run_prep(const DeltaArgs& a, hipStream_t s) {
  return launch(delta_prep_kernel<UT, EVEN, DK, ADJ>, static_cast<long long>(a.B) * a.HV * a.nc, 256, s, a);
}
// the scans' grid: every head's slices on one XCD
long long scan_grid(const DeltaArgs& a, int cols) { return ceil_div(static_cast<long long>(a.B) * a.HV, 8) * 8 * ceil_div(a.dv, cols); }

struct DeltaForward {
  template <class UT, int MODE, int DK>
  static int run(const DeltaArgs& a, const float*, float*, float*, hipStream_t s) {
    if (const int rc = run_prep<UT, MODE != kOdd, DK, false>(a, s)) return rc;
    return launch(delta_scan_kernel<UT, MODE, DK, 1, 4>, scan_grid(a, 64), DeltaScan<UT, MODE, DK, 1, 4, false>::THREADS, s, a);
  }
};
struct DeltaAdjoint {
  template <class UT, int MODE, int DK>
  static int run(DeltaArgs a, const float* dsT, float* ds0, float* dlam, hipStream_t s) {
    constexpr bool EVEN = MODE != kOdd;
    if (const int rc = run_prep<UT, EVEN, DK, true>(a, s)) return rc;
    a.s0 = dsT;
    a.sT = ds0;
    if (const int rc = launch(delta_back_kernel<UT, MODE, DK, 1, 4>, scan_grid(a, 64), DeltaScan<UT, MODE, DK, 1, 4, true>::THREADS, s, a))
      return rc;
    if (const int rc = launch(delta_grad_kernel<UT, EVEN, DK>, static_cast<long long>(a.B) * a.H * a.nc, 512, s, a)) return rc;
    if (!dlam) return PARARNN_OK;
    return launch(delta_dlam_kernel, a.HV, 256, s, static_cast<const float*>(a.dlam_part), a.lam, dlam, a.B * a.nc, a.c);
  }
};
// mode: of bf16 tensors, kDirect where their rows take 16-byte loads of whole chunks, kEven where they start
// at multiples of 4 bytes
template <class R>
int run_delta(const DeltaArgs& a, int mode, const pararnn_delta_opts* o, const float* dsT, float* ds0, float* dlam, hipStream_t s) {
  const bool small = o->dk <= 64;
  if (o->dtype != PARARNN_BF16)
    return small ? R::template run<float, kEven, 64>(a, dsT, ds0, dlam, s) : R::template run<float, kEven, 128>(a, dsT, ds0, dlam, s);
  if (mode == kDirect)
    return small ? R::template run<bf16, kDirect, 64>(a, dsT, ds0, dlam, s) : R::template run<bf16, kDirect, 128>(a, dsT, ds0, dlam, s);
  if (mode == kEven)
    return small ? R::template run<bf16, kEven, 64>(a, dsT, ds0, dlam, s) : R::template run<bf16, kEven, 128>(a, dsT, ds0, dlam, s);
  return small ? R::template run<bf16, kOdd, 64>(a, dsT, ds0, dlam, s) : R::template run<bf16, kOdd, 128>(a, dsT, ds0, dlam, s);
}
int delta_mode(const pararnn_view* q, const pararnn_view* k, const pararnn_view* v, const pararnn_delta_opts* o, size_t es) {
  auto all = [&](size_t bytes) {
    return rows_aligned(q, es, o->dk, bytes, o->B) && rows_aligned(k, es, o->dk, bytes, o->B) && rows_aligned(v, es, o->dv, bytes, o->B);
  };
  return all(16) ? kDirect : all(4) ? kEven : kOdd;
}

}  // namespace
}  // namespace pararnn

using namespace pararnn;

extern "C" int32_t pararnn_delta_workspace_bytes(int32_t adjoint, const pararnn_delta_opts* o, size_t* bytes) {
  if (!bytes || !delta_ok(o) || (adjoint != 0 && adjoint != 1)) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const DeltaSizes z = delta_sizes(o, adjoint);
  *bytes = z.frags + z.rows + (adjoint ? z.states + z.ys + z.part : 0);
  return PARARNN_OK;
}

extern "C" int32_t pararnn_delta_saved_bytes(const pararnn_delta_opts* o, size_t* bytes) {
  if (!bytes || !delta_ok(o)) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const DeltaSizes z = delta_sizes(o, false);
  *bytes = z.states + z.ys;
  return PARARNN_OK;
}

extern "C" int32_t pararnn_delta_scan(const pararnn_view* q, const pararnn_view* k, const pararnn_view* v,
                                      const pararnn_view* gates, const float* lam, const float* s0, void* o, float* sT,
                                      void* saved, void* ws, size_t ws_bytes, const pararnn_delta_opts* opts,
                                      void* stream) {
  if (!delta_ok(opts) || !views_ok(q, k, v, gates, opts) || !lam || !o || !ws) return PARARNN_EINVAL;
  if (!dtype_ok(opts->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = opts->dtype == PARARNN_BF16 ? 2 : 4;
  for (const void* p : {q->p, k->p, v->p, gates->p, static_cast<const void*>(o)})
    if (!aligned(p, es)) return PARARNN_EUNSUPPORTED;
  if (!aligned(lam, 4) || !aligned(s0, 4) || !aligned(sT, 4) || !aligned(opts->lengths, 4) || !aligned(ws, kAlign) ||
      !aligned(saved, kAlign))
    return PARARNN_EUNSUPPORTED;
  const DeltaSizes z = delta_sizes(opts, false);
  if (ws_bytes < z.frags + z.rows) return PARARNN_EWORKSPACE;
  DeltaArgs a;
  delta_fill(a, q, k, v, gates, lam, opts, es);
  a.s0 = s0;
  a.sT = sT;
  a.o = o;
  char* w = static_cast<char*>(ws);
  a.frags = reinterpret_cast<bf16x8*>(w);
  a.rows = reinterpret_cast<float*>(w + z.frags);
  if (saved) {
    a.states = static_cast<f32x4*>(saved);
    a.ys = reinterpret_cast<f32x4*>(static_cast<char*>(saved) + z.states);
  }
  const pararnn_view ov = {o, static_cast<int64_t>(opts->L) * opts->HV * opts->dv, static_cast<int64_t>(opts->HV) * opts->dv};
  a.wide = rows_aligned(&ov, es, opts->dv, 16, opts->B);
  return run_delta<DeltaForward>(a, delta_mode(q, k, v, opts, es), opts, nullptr, nullptr, nullptr, static_cast<hipStream_t>(stream));
}

extern "C" int32_t pararnn_delta_scan_adjoint(const pararnn_view* q, const pararnn_view* k, const pararnn_view* v,
                                              const pararnn_view* gates, const float* lam, const void* saved,
                                              const void* d_o, const float* dsT, const pararnn_view* dq,
                                              const pararnn_view* dk, const pararnn_view* dv,
                                              const pararnn_view* dgates, float* dlam, float* ds0, void* ws,
                                              size_t ws_bytes, const pararnn_delta_opts* opts, void* stream) {
  if (!delta_ok(opts) || !views_ok(q, k, v, gates, opts) || !views_ok(dq, dk, dv, dgates, opts) || !lam || !saved ||
      !d_o || !ws)
    return PARARNN_EINVAL;
  if (!dtype_ok(opts->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = opts->dtype == PARARNN_BF16 ? 2 : 4;
  for (const void* p : {q->p, k->p, v->p, gates->p, dq->p, dk->p, dv->p, dgates->p, d_o})
    if (!aligned(p, es)) return PARARNN_EUNSUPPORTED;
  if (!aligned(lam, 4) || !aligned(dsT, 4) || !aligned(ds0, 4) || !aligned(dlam, 4) || !aligned(opts->lengths, 4) ||
      !aligned(ws, kAlign) || !aligned(saved, kAlign))
    return PARARNN_EUNSUPPORTED;
  const DeltaSizes z = delta_sizes(opts, true);
  if (ws_bytes < z.frags + z.rows + z.states + z.ys + z.part) return PARARNN_EWORKSPACE;
  DeltaArgs a;
  delta_fill(a, q, k, v, gates, lam, opts, es);
  a.gq = view(dq);
  a.gk = view(dk);
  a.gv = view(dv);
  a.dgates = view(dgates);
  a.o = const_cast<void*>(d_o);
  const pararnn_view ov = {d_o, static_cast<int64_t>(opts->L) * opts->HV * opts->dv, static_cast<int64_t>(opts->HV) * opts->dv};
  a.wide = rows_aligned(dv, es, opts->dv, 16, opts->B);
  char* w = static_cast<char*>(ws);
  a.frags = reinterpret_cast<bf16x8*>(w);
  w += z.frags;
  a.rows = reinterpret_cast<float*>(w);
  w += z.rows;
  a.dstates = reinterpret_cast<f32x4*>(w);
  w += z.states;
  a.dxs = reinterpret_cast<f32x4*>(w);
  w += z.ys;
  a.dlam_part = dlam ? reinterpret_cast<float*>(w) : nullptr;
  a.states = static_cast<f32x4*>(const_cast<void*>(saved));
  a.ys = reinterpret_cast<f32x4*>(static_cast<char*>(const_cast<void*>(saved)) + z.states);
  return run_delta<DeltaAdjoint>(a, delta_mode(q, k, &ov, opts, es), opts, dsT, ds0, dlam, static_cast<hipStream_t>(stream));
}

extern "C" int32_t pararnn_delta_step(const pararnn_view* q, const pararnn_view* k, const pararnn_view* v,
                                      const pararnn_view* gates, const float* lam, const int32_t* slots, float* state,
                                      void* o, int32_t S, const pararnn_delta_opts* opts, void* stream) {
  if (!delta_ok(opts) || opts->L != 1 || !lam || !state || !o || S < 1 || (!slots && S < opts->B)) return PARARNN_EINVAL;
  const long long nk = static_cast<long long>(opts->H) * opts->dk, nv = static_cast<long long>(opts->HV) * opts->dv;
  for (const auto& x : {std::make_pair(q, nk), std::make_pair(k, nk), std::make_pair(v, nv), std::make_pair(gates, 2LL * opts->HV)})
    if (!x.first || !x.first->p || x.first->batch > (1LL << 50) || (opts->B > 1 && x.first->batch < x.second)) return PARARNN_EINVAL;
  if (!dtype_ok(opts->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = opts->dtype == PARARNN_BF16 ? 2 : 4;
  for (const void* p : {q->p, k->p, v->p, gates->p, static_cast<const void*>(o)})
    if (!aligned(p, es)) return PARARNN_EUNSUPPORTED;
  if (!aligned(lam, 4) || !aligned(slots, 4) || !aligned(state, 4)) return PARARNN_EUNSUPPORTED;
  DeltaStepArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q->p;
  a.k = k->p;
  a.v = v->p;
  a.gates = gates->p;
  a.q_row = q->batch;
  a.k_row = k->batch;
  a.v_row = v->batch;
  a.g_row = gates->batch;
  a.lam = lam;
  a.slots = slots;
  a.state = state;
  a.o = o;
  a.B = opts->B;
  a.H = opts->H;
  a.HV = opts->HV;
  a.dk = opts->dk;
  a.dv = opts->dv;
  a.S = S;
  a.c = opts->c;
  a.eps = opts->eps;
  a.scale = opts->scale;
  a.wide = opts->dv % 4 == 0 && aligned(state, 16);
  const long long grid = static_cast<long long>(opts->B) * opts->HV * ceil_div(opts->dv, 32);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (opts->dtype == PARARNN_BF16) return launch(delta_step_kernel<bf16>, grid, 256, st, a);
  return launch(delta_step_kernel<float>, grid, 256, st, a);
}
