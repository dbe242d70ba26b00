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
#include "delta/matmul_int8.h"
#include "delta/norm_block.h"
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
         // the largest launches: a chunk of all heads at once, and a scan's slices of all heads
         static_cast<long long>(o->B) * o->HV * ceil_div(o->L, kDeltaChunk) <= kMaxThreads / 512 &&
         (static_cast<long long>(o->B) * o->HV + 7) * ceil_div(o->dv, 64) <= kMaxThreads / 512;
}

// sizes of a call's pieces, in bytes (chunks of all value heads)
struct DeltaSizes {
  size_t frags, rows, states, ys, part, seg_add, seg_map;
};
// Segments that the scans cut a sequence into, and chunks of each: as many as give every CU a workgroup, and no
// more than make the product over the others' maps as long as the scan of the own chunks. A map takes as long as
// two chunks in bf16 and half a chunk in fp32: sqrt(0.8 chunks) and sqrt(4.5 chunks) (forward with factors 0.8, 1.6
// and 4.5: B = 1 L = 65536 H = 2 128 wide bf16 424, 514, 673 us, L = 1024 H = 1 64 wide fp32 71, 58, 47). The
// segments' scan before the scans pays from three of them on (bf16, B = 5 L = 4096 H = 8, three: 210 -> 188 us; two,
// B = 8: 234 -> 272), in the adjoint, which both scans are less of, from four on (three: 570 -> 584 us; B = 1 L =
// 4096 H = 32, four: 507 -> 500), and in bf16, whose chunks are passed in a third of fp32's time, from 16 chunks on
// (H = 8, 9 chunks: 37 -> 44 us, 16: 55 -> 56, 32 and B = 4: 106 -> 99; fp32, 6 chunks: 49 -> 38). B = 1 L = 65536
// H = 16: 2815 -> 1082 us (all measured with two planes in what goes to bf16 outputs; with three 1220).
struct DeltaSegments {
  int n, per;
};
DeltaSegments delta_segments(const pararnn_delta_opts* o, bool adj) {
  const long long nc = ceil_div(o->L, kDeltaChunk), groups = static_cast<long long>(o->B) * o->HV * ceil_div(o->dv, 64);
  const double share = o->dtype == PARARNN_BF16 ? 0.8 : 4.5;
  const long long most = static_cast<long long>(sqrt(share * static_cast<double>(nc))), room = kCUs / groups;
  const long long n = room < most ? room : most;
  if (n < (adj ? 4 : 3) || (o->dtype == PARARNN_BF16 && nc < 16)) return {1, static_cast<int>(nc)};
  const int per = static_cast<int>(ceil_div(nc, n));
  return {static_cast<int>(ceil_div(nc, per)), per};
}
DeltaSizes delta_sizes(const pararnn_delta_opts* o) {
  const size_t chunks = static_cast<size_t>(o->B) * o->HV * ceil_div(o->L, kDeltaChunk);
  // the forward pass's segments, which are the adjoint's or more: a workspace of the adjoint serves both
  const int DK = o->dk <= 64 ? 64 : 128, n = delta_segments(o, false).n;
  const size_t segs = n > 1 ? static_cast<size_t>(o->B) * o->HV * n : 0;
  return {round_up(chunks * DeltaFrags::ALL * sizeof(bf16x8)), round_up(chunks * kRows * 64 * sizeof(float)),
          chunks * delta_tiles(o->dv) * delta_tiles(o->dk) * 1024, chunks * delta_tiles(o->dv) * 4096,
          round_up(chunks * sizeof(float)), segs * delta_tiles(o->dv) * (DK / 16) * 1024, segs * DK * DK * 4};
}

size_t delta_bytes(const DeltaSizes& z, bool adj) {
  return z.frags + z.rows + z.seg_add + z.seg_map + (adj ? z.states + z.ys + z.part : 0);
}
// the workspace's pieces that both directions have; returns what follows them
char* delta_carve(DeltaArgs& a, void* ws, const DeltaSizes& z) {
  char* w = static_cast<char*>(ws);
  a.frags = reinterpret_cast<bf16x8*>(w);
  w += z.frags;
  a.rows = reinterpret_cast<float*>(w);
  w += z.rows;
  a.seg_add = reinterpret_cast<f32x4*>(w);
  w += z.seg_add;
  a.seg_map = reinterpret_cast<float*>(w);
  return w + z.seg_map;
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
                const pararnn_view* gates, const float* lam, const pararnn_delta_opts* o, bool adj) {
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
  const DeltaSegments g = delta_segments(o, adj);
  a.nseg = g.n;
  a.per = g.per;
}

template <class UT, bool EVEN, int DK, bool ADJ>
int run_prep(const DeltaArgs& a, hipStream_t s) {
  return launch(delta_prep_kernel<UT, EVEN, DK, ADJ>, static_cast<long long>(a.B) * a.HV * a.nc, 256, s, a);
}
// the scans' grid: every head's slices on one XCD
long long scan_grid(const DeltaArgs& a, long long slices) {
  return ceil_div(static_cast<long long>(a.B) * a.HV * a.nseg, 8) * 8 * slices;
}
template <class UT, int MODE, int DK, bool ADJ>
int run_segments(const DeltaArgs& a, hipStream_t s) {
  if (a.nseg == 1) return PARARNN_OK;
  // Forward, bf16 and more than 64 columns: 8 waves, for which 168 registers are enough, read a chunk once for 128
  // (B = 5 L = 1237 HV = 6: 34 -> 25 us; with 4 waves the matrix cores wait for each wave's chain)
  if constexpr (!ADJ && sizeof(UT) == 2 && DK == 128) {
    if (a.dv > 64)
      return launch(delta_segment_kernel<UT, MODE, DK, 1, 8, false>, scan_grid(a, ceil_div(a.dv, 128) + 1),
                    DeltaScan<UT, MODE, DK, 1, 8, false, true>::THREADS, s, a);
  }
  return launch(delta_segment_kernel<UT, MODE, DK, 1, 4, ADJ>, scan_grid(a, ceil_div(a.dv, 64) + ceil_div(a.dk, 64)),
                DeltaScan<UT, MODE, DK, 1, 4, ADJ, true>::THREADS, s, a);
}

// Few heads: half as many columns to a workgroup, on twice as many CUs (128 workgroups of 64: 301 us as 272, 30: 71 as 68)
bool narrow(const DeltaArgs& a) { return static_cast<long long>(a.B) * a.HV * a.nseg * ceil_div(a.dv, 64) <= kCUs / 2; }

struct DeltaForward {
  template <class UT, int MODE, int DK>
  static int run(const DeltaArgs& a, const float*, float*, float*, hipStream_t s) {
    if (const int rc = run_prep<UT, MODE != kOdd, DK, false>(a, s)) return rc;
    if (const int rc = run_segments<UT, MODE, DK, false>(a, s)) return rc;
    return narrow(a) ? launch(delta_scan_kernel<UT, MODE, DK, 1, 2>, scan_grid(a, ceil_div(a.dv, 32)), DeltaScan<UT, MODE, DK, 1, 2, false>::THREADS, s, a)
                     : launch(delta_scan_kernel<UT, MODE, DK, 1, 4>, scan_grid(a, ceil_div(a.dv, 64)), DeltaScan<UT, MODE, DK, 1, 4, false>::THREADS, s, a);
  }
};
struct DeltaAdjoint {
  template <class UT, int MODE, int DK>
  static int run(DeltaArgs a, const float* dsT, float* ds0, float* dlam, hipStream_t s) {
    constexpr bool EVEN = MODE != kOdd;
    if (const int rc = run_prep<UT, EVEN, DK, true>(a, s)) return rc;
    a.s0 = dsT;
    a.sT = ds0;
    if (const int rc = run_segments<UT, MODE, DK, true>(a, s)) return rc;
    if (const int rc = narrow(a) ? launch(delta_back_kernel<UT, MODE, DK, 1, 2>, scan_grid(a, ceil_div(a.dv, 32)), DeltaScan<UT, MODE, DK, 1, 2, true>::THREADS, s, a)
                                 : launch(delta_back_kernel<UT, MODE, DK, 1, 4>, scan_grid(a, ceil_div(a.dv, 64)), DeltaScan<UT, MODE, DK, 1, 4, true>::THREADS, s, a))
      return rc;
    const long long grid = static_cast<long long>(a.B) * a.H * a.nc;
    if (const int rc = a.H == a.HV ? launch(delta_grad_kernel<UT, EVEN, DK, false>, grid, 512, s, a)
                                   : launch(delta_grad_kernel<UT, EVEN, DK, true>, grid, 512, s, a))
      return rc;
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

// ---------------------------------------------------------------------------
// norms around a block

constexpr int kNormBlockMaxD = 16384;

bool norm_block_ok(const pararnn_norm_block_opts* o) {
  return o && o->N >= 1 && o->D >= 1 && o->D <= kNormBlockMaxD && o->group >= 1 && o->group <= o->D && o->D % o->group == 0 &&
         o->eps >= 0.0f && isfinite(o->eps) && o->x_row >= o->D && static_cast<double>(o->N) * o->D < 2.0e18 &&
         static_cast<double>(o->N) * static_cast<double>(o->x_row) < 2.0e18;
}

// Threads per row and vectors of 8 columns per thread: as few threads as have one vector each up to 2048 columns
// (twice as many: 4999 x 1000 9.3 -> 12.4 us, 262144 x 128 45 -> 49 us), two above, since a workgroup's sum waits for
// its last wave (4096 x 4096, 256 or 512 threads: 24 and 30 us; 4096 x 8192, 512 or 1024: 49 and 72). The adjoint,
// which holds four times the registers per column, has one up to 4096 columns (256 threads with two there: 66 ->
// 92 us), and above, with a residual (pre), whose three partial sums do not fit in 1024 threads' registers, two up
// to 8192 (126 us, 1024 threads 150; without a residual 62 and 56).
struct NormBlockShape {
  int tpr, nv;
};
NormBlockShape norm_block_shape(int D, bool adjoint, bool pre) {
  const int v = static_cast<int>(ceil_div(D, 8));
  for (int t : {16, 32, 64, 128, 256})
    if (v <= t) return {t, 1};
  if (adjoint && v <= 512) return {512, 1};
  if (adjoint && !pre && v <= 1024) return {1024, 1};
  return v <= 512 ? NormBlockShape{256, 2} : v <= 1024 ? NormBlockShape{512, 2} : NormBlockShape{1024, 2};
}
// workgroups of the adjoint: each leaves a partial row of every parameter, so no more than fill the CUs
long long norm_block_adjoint_grid(long long N, int D, bool pre) {
  const NormBlockShape k = norm_block_shape(D, true, pre);
  const long long rounds = ceil_div(N, k.tpr < 256 ? 256 / k.tpr : 1), room = kCUs * (k.tpr <= 256 ? 4 : 1024 / k.tpr);
  return rounds <= room ? rounds : room;
}

// A call's rows as the kernels take them: groups without a residual and with y in the input's type are rows
struct NormBlockRows {
  long long N;
  int D, H, lanes;
};
NormBlockRows norm_block_rows(const pararnn_norm_block_opts* o, bool residual, bool int8) {
  if (o->group == o->D) return {o->N, o->D, 1, 0};
  if (!residual && !int8) return {o->N * (o->D / o->group), o->group, o->D / o->group, 0};
  return {o->N, o->D, 1, o->group / 8};
}
// groups within a row: 8 columns times a power of two up to a wave's lanes
bool norm_block_group_ok(const pararnn_norm_block_opts* o, const NormBlockRows& r) {
  return r.D == o->group || (o->group % 8 == 0 && r.lanes <= 64 && (r.lanes & (r.lanes - 1)) == 0);
}

template <bool ADJ, bool PRE, class F>
int norm_block_dispatch(int D, F go) {
  const NormBlockShape k = norm_block_shape(D, ADJ, PRE);
#define PARARNN_SHAPE(T, V) \
  if (k.tpr == T && k.nv == V) return go(std::integral_constant<int, T>{}, std::integral_constant<int, V>{})
  PARARNN_SHAPE(16, 1);
  PARARNN_SHAPE(32, 1);
  PARARNN_SHAPE(64, 1);
  PARARNN_SHAPE(128, 1);
  PARARNN_SHAPE(256, 1);
  if constexpr (ADJ) {
    PARARNN_SHAPE(512, 1);
  } else {
    PARARNN_SHAPE(256, 2);
  }
  if constexpr (ADJ && !PRE) {
    PARARNN_SHAPE(1024, 1);
  } else {
    PARARNN_SHAPE(512, 2);
  }
#undef PARARNN_SHAPE
  return go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}
template <class XT, bool PRE, bool INT8, bool ALIGNED>
int launch_norm_block(const NormBlockArgs& a, bool stream, hipStream_t s) {
  return norm_block_dispatch<false, PRE>(a.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    long long grid = ceil_div(a.N, TPR < 256 ? 256 / TPR : 1);
    if (grid > 8192) grid = 8192;
    const int block = TPR < 256 ? 256 : TPR;
    if (ALIGNED && stream) return launch(norm_block_kernel<XT, TPR, NV, PRE, INT8, ALIGNED, ALIGNED>, grid, block, s, a);
    return launch(norm_block_kernel<XT, TPR, NV, PRE, INT8, ALIGNED, false>, grid, block, s, a);
  });
}
template <class XT, bool PRE, bool ALIGNED>
int launch_norm_block_adjoint(const NormBlockArgs& a, long long grid, bool stream, hipStream_t s) {
  return norm_block_dispatch<true, PRE>(a.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    const int block = TPR < 256 ? 256 : TPR;
    if (ALIGNED && stream) return launch(norm_block_adjoint_kernel<XT, TPR, NV, PRE, ALIGNED, ALIGNED>, grid, block, s, a);
    return launch(norm_block_adjoint_kernel<XT, TPR, NV, PRE, ALIGNED, false>, grid, block, s, a);
  });
}
// every row of 8-column vectors starts at a multiple of 16 bytes
bool norm_block_aligned(const NormBlockRows& r, size_t es, std::initializer_list<const void*> ptrs,
                        std::initializer_list<long long> strides) {
  bool ok = r.D % 8 == 0;
  for (const void* q : ptrs) ok = ok && (!q || aligned(q, 16));
  for (long long t : strides) ok = ok && t * es % 16 == 0;
  return ok;
}

// ---------------------------------------------------------------------------
// 8-bit integer product

typedef MatmulShape<2, 2, 4, 4, 1> Int8Mid;
typedef MatmulShape<2, 2, 2, 2, 1> Int8Small;
typedef MatmulShape<2, 2, 2, 2, 2> Int8Split2;
typedef MatmulShape<2, 2, 2, 2, 4> Int8Split4;

// Which large tile: 256 x 256 (4), 256 x 192 (3), or neither (0), by the rounds over the CUs and the steps of a
// round (measured, 256 x 256, 256 x 192 and 128 x 128: 32768 x 16384 x 4096 1789, 1924, 2005 us; 6000 x 6000 x 3968
// 158, 132, 140; 2048 x 4096 x 4096 51, 43, 33; 8192 x 5120 x 2048, where it misses the best by 6%, 94, 99, 89)
int int8_large_tile(const Int8Args& p) {
  const long long tm = ceil_div(p.M, 256);
  const double kb = p.KB;
  const double mid = ceil_div(ceil_div(p.M, 128) * ceil_div(p.N, 128), 2 * kCUs) * (2.7 * kb + 14.0);
  const double l4 = ceil_div(tm * ceil_div(p.N, 256), kCUs) * (4.0 * kb + 20.0);
  const double l3 = ceil_div(tm * ceil_div(p.N, 192), kCUs) * (3.0 * kb + 20.0);
  if (mid < l4 && mid < l3) return 0;
  return l4 <= l3 ? 4 : 3;
}
template <class S, bool F32OUT>
int launch_int8(const Int8Args& p, bool direct, hipStream_t s) {
  const long long grid = ceil_div(p.M, S::BM) * ceil_div(p.N, S::BN);
  return direct ? launch(int8_kernel<S, F32OUT, true>, grid, S::NT * S::KS, s, p)
                : launch(int8_kernel<S, F32OUT, false>, grid, S::NT * S::KS, s, p);
}
template <bool F32OUT, int MT, int NT, int UN>
int launch_int8_few(const Int8Args& p, hipStream_t s) {
  return launch(int8_few_kernel<F32OUT, MT, NT, UN>, ceil_div(p.N, 16 * NT), 512, s, p);
}
template <bool F32OUT>
int launch_int8_shape(const Int8Args& p, bool direct, hipStream_t s) {
  const long long n16 = ceil_div(p.N, 16);
  // Up to 32 rows w goes from memory straight into registers, as wide a piece for each workgroup as leaves every CU
  // one (16 x 16384 x 4096, 64, 32 or 16 columns: 12.7, 15.7, 17.8 us, in tiles 15.2; 16 x 4096: 10.9, 7.8, 6.0, 8.3;
  // 64 rows, 2048 x 4096: 11.1, in tiles 8.4)
  if (direct && p.M <= 32) {
    if (n16 >= 3 * kCUs) return p.M <= 16 ? launch_int8_few<F32OUT, 1, 4, 1>(p, s) : launch_int8_few<F32OUT, 2, 4, 1>(p, s);
    if (n16 >= 2 * kCUs) return p.M <= 16 ? launch_int8_few<F32OUT, 1, 2, 2>(p, s) : launch_int8_few<F32OUT, 2, 2, 2>(p, s);
    return p.M <= 16 ? launch_int8_few<F32OUT, 1, 1, 4>(p, s) : launch_int8_few<F32OUT, 2, 1, 2>(p, s);
  }
  const int tn = direct ? int8_large_tile(p) : 0;
  if (tn == 4) return launch(int8_large_kernel<4, F32OUT>, ceil_div(p.M, 256) * ceil_div(p.N, 256), 512, s, p);
  if (tn == 3) return launch(int8_large_kernel<3, F32OUT>, ceil_div(p.M, 256) * ceil_div(p.N, 192), 512, s, p);
  // 128 x 128 tiles from one per CU on (2048 x 4096 x 4096: 33 us, 64 x 64 48; 1024 rows: 27 and 25)
  if (ceil_div(p.M, 128) * ceil_div(p.N, 128) >= kCUs) return launch_int8<Int8Mid, F32OUT>(p, direct, s);
  // few tiles: K dealt out to groups of waves (256 x 4096 x 4096, one, two or four: 12.4, 10.3, 10.0 us; 512 rows:
  // 16.8, 15.3, 20.3; 1024: 25, 28, 39; 300 x 1000 x 512: 4.0, 4.1, 4.5)
  const long long tiles = ceil_div(p.M, 64) * ceil_div(p.N, 64);
  if (direct && tiles <= kCUs && p.KB >= 8) return launch_int8<Int8Split4, F32OUT>(p, true, s);
  if (tiles <= 2 * kCUs && p.KB >= 8) return launch_int8<Int8Split2, F32OUT>(p, direct, s);
  return launch_int8<Int8Small, F32OUT>(p, direct, s);
}

}  // namespace
}  // namespace pararnn

using namespace pararnn;

extern "C" int32_t pararnn_delta_workspace_bytes(int32_t adjoint, const pararnn_delta_opts* o, size_t* bytes) {
  if (!bytes || !delta_ok(o) || (adjoint != 0 && adjoint != 1)) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const DeltaSizes z = delta_sizes(o);
  *bytes = delta_bytes(z, adjoint);
  return PARARNN_OK;
}

extern "C" int32_t pararnn_delta_saved_bytes(const pararnn_delta_opts* o, size_t* bytes) {
  if (!bytes || !delta_ok(o)) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const DeltaSizes z = delta_sizes(o);
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
  const DeltaSizes z = delta_sizes(opts);
  if (ws_bytes < delta_bytes(z, false)) return PARARNN_EWORKSPACE;
  DeltaArgs a;
  delta_fill(a, q, k, v, gates, lam, opts, false);
  a.s0 = s0;
  a.sT = sT;
  a.o = o;
  delta_carve(a, ws, z);
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
  const DeltaSizes z = delta_sizes(opts);
  if (ws_bytes < delta_bytes(z, true)) return PARARNN_EWORKSPACE;
  DeltaArgs a;
  delta_fill(a, q, k, v, gates, lam, opts, true);
  a.gq = view(dq);
  a.gk = view(dk);
  a.gv = view(dv);
  a.dgates = view(dgates);
  a.o = const_cast<void*>(d_o);
  const pararnn_view ov = {d_o, static_cast<int64_t>(opts->L) * opts->HV * opts->dv, static_cast<int64_t>(opts->HV) * opts->dv};
  a.wide = rows_aligned(dv, es, opts->dv, 16, opts->B);
  a.wide_qk = opts->dk % 8 == 0 && rows_aligned(dq, es, opts->dk, 16, opts->B) && rows_aligned(dk, es, opts->dk, 16, opts->B);
  char* w = delta_carve(a, ws, z);
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

extern "C" int32_t pararnn_norm_block(const void* x, const void* gate, const void* residual, const float* w,
                                      const float* alpha, const float* w_next, void* s, void* y, float* scale,
                                      const pararnn_norm_block_opts* o, void* stream_) {
  if (!norm_block_ok(o) || !x || !y || (!w && !residual)) return PARARNN_EINVAL;
  if (residual ? !w_next || !s || o->residual_row < o->D : alpha || w_next || s) return PARARNN_EINVAL;
  if (gate && o->gate_row < o->D) return PARARNN_EINVAL;
  if (o->out != PARARNN_NORM_BLOCK_SAME && o->out != PARARNN_NORM_BLOCK_INT8) return PARARNN_EINVAL;
  const bool int8 = o->out == PARARNN_NORM_BLOCK_INT8;
  if (int8 && !scale) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = o->dtype == PARARNN_BF16 ? 2 : 4;
  for (const void* p : {x, gate, residual, static_cast<const void*>(s)})
    if (!aligned(p, es)) return PARARNN_EUNSUPPORTED;
  if ((!int8 && !aligned(y, es)) || !aligned(w, 4) || !aligned(alpha, 4) || !aligned(w_next, 4) || !aligned(scale, 4))
    return PARARNN_EUNSUPPORTED;
  const NormBlockRows r = norm_block_rows(o, residual, int8);
  if (w && !norm_block_group_ok(o, r)) return PARARNN_EUNSUPPORTED;
  NormBlockArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.gate = gate;
  a.residual = residual;
  a.w = w;
  a.alpha = alpha;
  a.w_next = w_next;
  a.s = s;
  a.y = y;
  a.scale = scale;
  a.N = r.N;
  a.D = r.D;
  a.H = r.H;
  a.lanes = w ? r.lanes : 0;
  a.G = o->group;
  a.x_row = o->x_row;
  a.gate_row = o->gate_row;
  a.residual_row = o->residual_row;
  a.eps = o->eps;
  hipStream_t st = static_cast<hipStream_t>(stream_);
  const bool ok = norm_block_aligned(r, es, {x, gate, residual, s, y, w, alpha, w_next},
                                     {o->x_row, gate ? o->gate_row : 0, residual ? o->residual_row : 0});
  // past the caches where the tensors together are larger than the last-level one (2048 columns, past them and
  // through them: 230 MB 38.9 and 36.0 us, 307 MB 52.1 and 56.4)
  const bool far = static_cast<double>(o->N) * o->D * es * (2 + (gate != nullptr) + 2 * (residual != nullptr)) > 256.0 * 1024 * 1024;
  auto go = [&](auto xt, auto aligned_) {
    typedef decltype(xt) XT;
    constexpr bool AL = decltype(aligned_)::value;
    if (residual) return int8 ? launch_norm_block<XT, true, true, AL>(a, far, st) : launch_norm_block<XT, true, false, AL>(a, far, st);
    return int8 ? launch_norm_block<XT, false, true, AL>(a, far, st) : launch_norm_block<XT, false, false, AL>(a, far, st);
  };
  if (o->dtype == PARARNN_BF16) return ok ? go(bf16{}, std::true_type{}) : go(bf16{}, std::false_type{});
  return ok ? go(0.0f, std::true_type{}) : go(0.0f, std::false_type{});
}

extern "C" int32_t pararnn_norm_block_workspace_bytes(const pararnn_norm_block_opts* o, int32_t residual, size_t* bytes) {
  if (!norm_block_ok(o) || !bytes) return PARARNN_EINVAL;
  const NormBlockRows r = norm_block_rows(o, residual != 0, false);
  *bytes = round_up(sizeof(float) * static_cast<size_t>(norm_block_adjoint_grid(r.N, r.D, residual)) * (residual ? 3 : 1) * r.D);
  return PARARNN_OK;
}

extern "C" int32_t pararnn_norm_block_adjoint(const void* x, const void* gate, const void* s, const float* w,
                                              const float* alpha, const float* w_next, const void* dy, const void* ds,
                                              void* dx, void* dgate, void* dresidual, float* dw, float* dalpha,
                                              float* dw_next, void* ws, size_t ws_bytes,
                                              const pararnn_norm_block_opts* o, void* stream_) {
  if (!norm_block_ok(o) || !x || !dy || !dx || (!w && !s) || (gate != nullptr) != (dgate != nullptr)) return PARARNN_EINVAL;
  if (s ? !w_next || !dresidual : alpha || w_next || ds || dresidual || dalpha || dw_next) return PARARNN_EINVAL;
  if ((gate && o->gate_row < o->D) || (dw && !w)) return PARARNN_EINVAL;
  const bool sums = dw || dalpha || dw_next;
  if (sums && !ws) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = o->dtype == PARARNN_BF16 ? 2 : 4;
  for (const void* p : {x, gate, s, dy, ds, static_cast<const void*>(dx), static_cast<const void*>(dgate),
                        static_cast<const void*>(dresidual)})
    if (!aligned(p, es)) return PARARNN_EUNSUPPORTED;
  for (const void* p : {static_cast<const void*>(w), static_cast<const void*>(alpha), static_cast<const void*>(w_next),
                        static_cast<const void*>(dw), static_cast<const void*>(dalpha), static_cast<const void*>(dw_next)})
    if (!aligned(p, 4)) return PARARNN_EUNSUPPORTED;
  const NormBlockRows r = norm_block_rows(o, s != nullptr, false);
  if (w && !norm_block_group_ok(o, r)) return PARARNN_EUNSUPPORTED;
  const long long grid = norm_block_adjoint_grid(r.N, r.D, s != nullptr);
  const int parts = s ? 3 : 1;
  if (sums && ws_bytes < sizeof(float) * static_cast<size_t>(grid) * parts * r.D) return PARARNN_EWORKSPACE;
  if (sums && !aligned(ws, kAlign)) return PARARNN_EUNSUPPORTED;
  NormBlockArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.gate = gate;
  a.residual = s;
  a.w = w;
  a.alpha = alpha;
  a.w_next = w_next;
  a.dy = dy;
  a.ds = ds;
  a.dx = dx;
  a.dgate = dgate;
  a.dresidual = dresidual;
  a.part = sums ? static_cast<float*>(ws) : nullptr;
  a.N = r.N;
  a.D = r.D;
  a.H = r.H;
  a.lanes = w ? r.lanes : 0;
  a.G = o->group;
  a.x_row = o->x_row;
  a.gate_row = o->gate_row;
  a.eps = o->eps;
  hipStream_t st = static_cast<hipStream_t>(stream_);
  const bool ok = norm_block_aligned(r, es, {x, gate, s, dy, ds, dx, dgate, dresidual, w, alpha, w_next},
                                     {o->x_row, gate ? o->gate_row : 0});
  // as forward (2048 columns without a residual, past the caches and through them: 256 MB 58.9 and 53.0 us, 320 MB
  // 67.9 and 72.3; with one within 3% on both sides)
  const bool far = static_cast<double>(o->N) * o->D * es * (3 + 2 * (gate != nullptr) + 2 * (s != nullptr) + (ds != nullptr)) > 256.0 * 1024 * 1024;
  auto go = [&](auto xt, auto aligned_) {
    typedef decltype(xt) XT;
    constexpr bool AL = decltype(aligned_)::value;
    return s ? launch_norm_block_adjoint<XT, true, AL>(a, grid, far, st) : launch_norm_block_adjoint<XT, false, AL>(a, grid, far, st);
  };
  int rc;
  if (o->dtype == PARARNN_BF16) rc = ok ? go(bf16{}, std::true_type{}) : go(bf16{}, std::false_type{});
  else rc = ok ? go(0.0f, std::true_type{}) : go(0.0f, std::false_type{});
  if (rc || !sums) return rc;
  hipLaunchKernelGGL(norm_block_sum_kernel, dim3(static_cast<unsigned>(ceil_div(r.D, 32)), parts), dim3(1024), 0, st,
                     static_cast<const float*>(a.part), dw, dalpha, dw_next, grid, parts, r.D, o->group == o->D ? r.D : o->group);
  return check_hip(hipGetLastError());
}

extern "C" int32_t pararnn_matmul_int8(const void* a, const float* sa, const void* w, const float* sw, const float* bias,
                                       void* y, const pararnn_int8_opts* o, void* stream_) {
  if (!o || o->M < 1 || o->N < 1 || o->K < 1 || o->K > 131071 || !a || !sa || !w || !sw || !y) return PARARNN_EINVAL;
  if (o->M > 2147483647 - 256 || o->N > 2147483647 - 256) return PARARNN_EINVAL;
  if (static_cast<double>(ceil_div(o->M, 64)) * ceil_div(o->N, 64) > 2.0e9) return PARARNN_EINVAL;
  if (!dtype_ok(o->y_dtype)) return PARARNN_EUNSUPPORTED;
  const bool f32 = o->y_dtype == PARARNN_F32;
  if (!aligned(sa, 4) || !aligned(sw, 4) || !aligned(bias, 4) || !aligned(y, f32 ? 4 : 2)) return PARARNN_EUNSUPPORTED;
  Int8Args p;
  p.a = static_cast<const uint8_t*>(a);
  p.sa = sa;
  p.w = static_cast<const uint8_t*>(w);
  p.sw = sw;
  p.bias = bias;
  p.y = y;
  p.M = o->M;
  p.N = o->N;
  p.K = o->K;
  p.KB = static_cast<int>(ceil_div(o->K, 128));
  p.vec = !f32 && o->N % 8 == 0 && o->N <= (1 << 22) && aligned(y, 16) ? 8 : o->N % 4 == 0 && aligned(y, f32 ? 16 : 8) ? 4 : 1;
  // y past the caches where it is larger than the last one (16384 x 8192, K = 1024, 256 MB: 177 us, through them
  // 165; 16384 x 16384: 308 and 387)
  p.stream = 2.0 * p.M * p.N > 256.0 * 1024 * 1024;
  const bool direct = o->K % 16 == 0 && aligned(a, 16) && aligned(w, 16);
  hipStream_t s = static_cast<hipStream_t>(stream_);
  return f32 ? launch_int8_shape<true>(p, direct, s) : launch_int8_shape<false>(p, direct, s);
}
