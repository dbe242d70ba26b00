// layer.hip -- host side of the C ABI declared in include/pararnn_layer.h:
// argument checks, the choice of a launch shape, workspace carving and the
// launches, all asynchronous on the caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <type_traits>

#include "../../include/pararnn_layer.h"
#include "layer/gated_scan.h"
#include "layer/matmul_fp8.h"
#include "layer/norm.h"

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

// Launch shapes: C channels per lane, T steps per lane, LL lane groups, W
// waves, OCC waves per SIMD that the registers must allow
template <class UT, int C> struct ScanShape;
template <> struct ScanShape<bf16, 2> { static constexpr int T = 12, LL = 2, W = 8, OCC = 5; };
template <> struct ScanShape<bf16, 1> { static constexpr int T = 16, LL = 1, W = 8, OCC = 4; };
template <> struct ScanShape<float, 2> { static constexpr int T = 8, LL = 4, W = 8, OCC = 4; };
template <> struct ScanShape<float, 1> { static constexpr int T = 16, LL = 2, W = 8, OCC = 4; };
template <int C> struct AdjShape { static constexpr int T = 6, LL = 2, W = 8, OCC = 4; };
template <> struct AdjShape<1> { static constexpr int T = 12, LL = 1, W = 8, OCC = 4; };

// Small problems, where latency counts: the whole sequence in one workgroup of
// 16 waves, so that there is no carry between chunks, nothing to clear and one
// launch per pass. It reads only 4 C channels of a row.
struct SmallShape { static constexpr int T = 4, LL = 16, W = 16, OCC = 4; };
constexpr int kSmallSteps = SmallShape::T * SmallShape::LL * SmallShape::W;
// B * D up to which it is taken. 1024 steps, forward and adjoint, against chunks with their clear (fp32,
// on the device): 64 channels 5.8 and 11.1 us against 8.9 and 13.8, 256 6.7 and 15.6 against 9.2 and
// 14.3, 512 9.3 and 21.2 against 9.4 and 15.0, 1024 18 and 30 against 10 and 16 (every line of HBM is
// read by 8 workgroups). In bf16 the adjoint's side turns earlier (128 channels 11.6 against 12.1, 256
// 16.7 against 12.5), and up to 96 steps, one chunk, it is 10 against 7 us.
constexpr int kSmallChannels = 256;
bool gated_small(const pararnn_gated_opts* o) {
  return o->L <= kSmallSteps && static_cast<long long>(o->B) * o->D <= kSmallChannels;
}

struct ScanGeo {
  int chunk, cw;
};
template <class K, int C> constexpr ScanGeo geo_of() { return {K::T * K::LL * K::W, 64 / K::LL * C}; }
constexpr int kScanMaxC = 2;
ScanGeo scan_geo(const pararnn_gated_opts* o, int C, bool adj) {
  const bool h = o->dtype == PARARNN_BF16;
  if (gated_small(o)) return C == 2 ? geo_of<SmallShape, 2>() : geo_of<SmallShape, 1>();
  if (adj) return C == 2 ? geo_of<AdjShape<2>, 2>() : geo_of<AdjShape<1>, 1>();
  if (C == 2) return h ? geo_of<ScanShape<bf16, 2>, 2>() : geo_of<ScanShape<float, 2>, 2>();
  return h ? geo_of<ScanShape<bf16, 1>, 1>() : geo_of<ScanShape<float, 1>, 1>();
}
constexpr int kMaxScanChunk = kSmallSteps;
// Ticket counters: 8 for up to this many tickets, else 2. 8 keep the
// workgroups that start together from queueing at one counter (5 x 1237 x 1000
// 29 -> 24 us forward, 51 -> 42 us back); where many rounds follow each other
// that is a small share, and 2 runs keep neighbouring channels together
// (1 x 65536 x 2048: 230 and 418 us against 240 and 438).
constexpr long long kFewTickets = 3072;

// Chunks per group (chunk_carry): with many tiles per chunk row the chunk
// before has long finished when this one asks, and plain hand-over from chunk
// to chunk is the least work; with few, the chain of waits counts.
int gated_group(long long tiles_per_row) {
  return tiles_per_row >= 128 ? 1 : tiles_per_row >= 64 ? 2 : tiles_per_row >= 16 ? 4 : kMaxGroup;
}

struct GatedLayout {
  size_t ctr = 0, carry = 0, agg = 0, clear_end = 0, part = 0, total = 0;
  int nchunks = 0, ntiles_d = 0, group = 1, parts_log2 = 0;
  bool direct = false;  // a channel's steps are all in one workgroup: it writes dlam itself
};

GatedLayout gated_layout(const pararnn_gated_opts* o, bool adj, int C) {
  GatedLayout y;
  const ScanGeo g = scan_geo(o, C, adj);
  y.nchunks = static_cast<int>(ceil_div(o->L, g.chunk));
  y.ntiles_d = static_cast<int>(ceil_div(o->D, g.cw));
  const size_t slots = static_cast<size_t>(o->B) * y.ntiles_d * g.cw;
  y.group = gated_group(static_cast<long long>(o->B) * y.ntiles_d);
  y.direct = adj && y.nchunks * static_cast<long long>(o->B) == 1;
  size_t off = 0;
  const long long ntiles = static_cast<long long>(o->B) * y.ntiles_d;
  while (y.parts_log2 < (ntiles * y.nchunks <= kFewTickets ? 3 : 1) && (1 << y.parts_log2) < ntiles) ++y.parts_log2;
  if (y.nchunks > 1) {
    off = round_up(sizeof(uint32_t) * (kTicketStride << y.parts_log2));
    y.carry = off;
    off = round_up(off + sizeof(uint64_t) * slots * (ceil_div(y.nchunks, y.group) + 1));
    y.agg = off;
    if (y.group > 1) off = round_up(off + sizeof(uint64_t) * slots * 2 * y.nchunks);
  }
  y.clear_end = off;
  y.part = off;
  if (adj && !y.direct) off = round_up(off + sizeof(float) * y.nchunks * static_cast<size_t>(o->B) * o->D);
  y.total = off;
  return y;
}

bool gated_ok(const pararnn_gated_opts* o, bool adj) {
  if (!o || o->B < 1 || o->L < 1 || o->D < 1) return false;
  if (!(o->c > 0.0f) || !isfinite(o->c)) return false;
  if (o->L > 2147483647 - 2 * kMaxScanChunk) return false;  // step numbers of a last partial chunk
  if (static_cast<double>(o->B) * o->L * o->D * 12 > 9.0e18) return false;
  for (int C = 1; C <= kScanMaxC; C *= 2) {
    const ScanGeo g = scan_geo(o, C, adj);
    // workgroups of 512 threads, two equal runs of tiles (as many tickets as this have two counters)
    const long long tiles = static_cast<long long>(o->B) * ceil_div(o->D, g.cw);
    const double wgs = static_cast<double>(tiles == 1 ? 1 : tiles + tiles % 2) * ceil_div(o->L, g.chunk);
    if (wgs > static_cast<double>(kMaxThreads / 512)) return false;
  }
  // one chunk is addressed with 32-bit offsets below 2^31
  return static_cast<double>(kMaxScanChunk) * 3 * o->D * 4 < 2147483648.0;
}
bool dtype_ok(int dtype) { return dtype == PARARNN_F32 || dtype == PARARNN_BF16; }

template <class UT, int C, bool RST>
int launch_gated(const GatedArgs& a, bool adj, bool small, hipStream_t s) {
  const long long grid = static_cast<long long>(a.B) * a.ntiles_d;
  const long long all = (static_cast<long long>(a.run) << a.parts_log2) * a.nchunks;
  const GatedArgs& b = a;
  if (small) {
    using K = SmallShape;
    return adj ? launch(gated_adjoint_kernel<UT, C, K::T, K::W, K::LL, K::OCC, RST, true>, grid, 64 * K::W, s, b)
               : launch(gated_scan_kernel<UT, C, K::T, K::W, K::LL, K::OCC, RST, true>, grid, 64 * K::W, s, b);
  }
  if (adj) {
    using K = AdjShape<C>;
    return launch(gated_adjoint_kernel<UT, C, K::T, K::W, K::LL, K::OCC, RST, false>, all, 64 * K::W, s, b);
  }
  using K = ScanShape<UT, C>;
  static_assert(K::T * K::LL * K::W <= kMaxScanChunk && kGatedSave % K::T == 0, "chunk");
  // document starts take registers of their own
  return launch(gated_scan_kernel<UT, C, K::T, K::W, K::LL, RST ? 4 : K::OCC, RST, false>, all, 64 * K::W, s, b);
}
template <class UT>
int launch_gated_c(int C, const GatedArgs& a, bool adj, bool small, hipStream_t s) {
  const bool r = a.reset != nullptr;
  if (C == 2) return r ? launch_gated<UT, 2, true>(a, adj, small, s) : launch_gated<UT, 2, false>(a, adj, small, s);
  return r ? launch_gated<UT, 1, true>(a, adj, small, s) : launch_gated<UT, 1, false>(a, adj, small, s);
}

int gated(bool adj, GatedArgs& a, float* dlam, void* ws, size_t ws_bytes, const pararnn_gated_opts* o, int C,
          hipStream_t stream) {
  const GatedLayout y = gated_layout(o, adj, C);
  if (y.total && !ws) return PARARNN_EINVAL;
  if (ws_bytes < y.total) return PARARNN_EWORKSPACE;
  if (!aligned(ws, kAlign)) return PARARNN_EUNSUPPORTED;
  char* w = static_cast<char*>(ws);
  a.lengths = o->lengths;
  a.reset = o->reset;
  a.carry = reinterpret_cast<unsigned long long*>(w + y.carry);
  a.agg = reinterpret_cast<unsigned long long*>(w + y.agg);
  a.ctr = reinterpret_cast<unsigned int*>(w + y.ctr);
  if (dlam && y.direct) a.dlam = dlam;
  else if (dlam) a.dl_part = reinterpret_cast<float*>(w + y.part);
  a.B = o->B;
  a.L = o->L;
  a.D = o->D;
  a.nchunks = y.nchunks;
  a.ntiles_d = y.ntiles_d;
  a.group = y.group;
  a.parts_log2 = y.parts_log2;
  a.run = static_cast<unsigned>(ceil_div(static_cast<long long>(o->B) * y.ntiles_d, 1 << y.parts_log2));
  a.by_run = fast_div(a.run);
  a.by_row = fast_div(static_cast<unsigned>(y.ntiles_d));
  a.c = o->c;
  if (y.clear_end) {
    const int rc = clear(w, y.clear_end, stream);
    if (rc) return rc;
  }
  const bool small = gated_small(o);
  const int rc = o->dtype == PARARNN_BF16 ? launch_gated_c<bf16>(C, a, adj, small, stream)
                                          : launch_gated_c<float>(C, a, adj, small, stream);
  if (rc || !dlam || y.direct) return rc;
  return launch(column_sum_kernel, ceil_div(o->D, kSumCols), kSumCols * kSumGroups, stream,
                static_cast<const float*>(a.dl_part), dlam, static_cast<long long>(y.nchunks) * o->B,
                static_cast<int>(o->D), a.lam, o->c);
}

// ---------------------------------------------------------------------------
// norm

constexpr int kNormMaxD = 16384;

// Threads per row (tpr), 8-column vectors per thread (nv): a wave per row
// while its vectors fit 4 per lane, then a workgroup per row
struct NormShape {
  int tpr, nv;
};
NormShape norm_shape(int D) {
  if (D <= 512) return {64, 1};
  if (D <= 1024) return {64, 2};
  if (D <= 2048) return {256, 1};
  if (D <= 4096) return {256, 2};
  if (D <= 8192) return {512, 2};
  return {1024, 2};
}
int norm_rows(int tpr) { return tpr < 256 ? 256 / tpr : 1; }

// Workgroups of the adjoint, each of which leaves one partial row of dw: what
// the CUs hold at once (4 waves per SIMD; 32768 x 4096 takes 307 us with half
// as many, 205 with all), evenly where that is between one and two rounds (4999 x 1000: 14.5 ->
// 13.3 us)
long long norm_adjoint_grid(const pararnn_norm_opts* o) {
  const NormShape k = norm_shape(o->D);
  const long long rounds = ceil_div(o->N, norm_rows(k.tpr)), room = kCUs * 16 / (k.tpr < 256 ? 4 : k.tpr / 64);
  return rounds <= room ? rounds : rounds < 2 * room ? ceil_div(rounds, 2) : room;
}

// Tensors that together are larger than the last-level cache are read and
// written past it (32768 x 4096 to 8 bits: 173 -> 161 us); smaller ones may be
// there from the operator before, and are for the one behind.
bool norm_stream(const pararnn_norm_opts* o, int bytes_per_element) {
  return static_cast<double>(o->N) * o->D * bytes_per_element >= 256.0 * 1024 * 1024;
}

bool norm_ok(const pararnn_norm_opts* o) {
  return o && o->N >= 1 && o->D >= 1 && o->D <= kNormMaxD && o->eps >= 0.0f && isfinite(o->eps) &&
         static_cast<double>(o->N) * o->D < 2.0e18;
}

template <class XT, bool VEC, class F>
int norm_dispatch(int D, F go) {
  const NormShape k = norm_shape(D);
  if (k.tpr == 64) return k.nv == 1 ? go(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{})
                                    : go(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (k.tpr == 256) {
    if (k.nv == 1) return go(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    return go(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  }
  if (k.tpr == 512) return go(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

template <class XT, int OUT, bool VEC>
int launch_norm(const NormArgs& a, bool stream, hipStream_t s) {
  return norm_dispatch<XT, VEC>(a.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    long long grid = ceil_div(a.N, TPR < 256 ? 256 / TPR : 1);
    if (grid > 8192) grid = 8192;
    const int block = TPR < 256 ? 256 : TPR;
    return stream && VEC ? launch(norm_kernel<XT, TPR, NV, OUT, VEC, VEC>, grid, block, s, a)
                         : launch(norm_kernel<XT, TPR, NV, OUT, VEC, false>, grid, block, s, a);
  });
}
template <class XT, bool VEC>
int launch_norm_out(int out, const NormArgs& a, bool stream, hipStream_t s) {
  return out == kNormSame  ? launch_norm<XT, kNormSame, VEC>(a, stream, s)
         : out == kNormFp8 ? launch_norm<XT, kNormFp8, VEC>(a, stream, s)
                           : launch_norm<XT, kNormFp8Pow2, VEC>(a, stream, s);
}
template <class XT, bool VEC>
int launch_norm_adjoint(const NormArgs& a, long long grid, bool stream, hipStream_t s) {
  return norm_dispatch<XT, VEC>(a.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    const int block = TPR < 256 ? 256 : TPR;
    return stream && VEC ? launch(norm_adjoint_kernel<XT, TPR, NV, VEC, VEC>, grid, block, s, a)
                         : launch(norm_adjoint_kernel<XT, TPR, NV, VEC, false>, grid, block, s, a);
  });
}

// rows of 8-column vectors that every pointer is 16-byte aligned for
bool norm_vec(int D, std::initializer_list<const void*> ptrs) {
  bool ok = D % 8 == 0;
  for (const void* q : ptrs) ok = ok && (!q || aligned(q, 16));
  return ok;
}

// ---------------------------------------------------------------------------
// 8-bit product

// 128 x 128 of y by 4 waves (64 x 64 each), 64 x 64 by 4 (32 x 32 each), and
// the same with the blocks of K dealt out to 2 or 4 such groups
typedef MatmulShape<2, 2, 4, 4, 1> MatmulMid;
typedef MatmulShape<2, 2, 2, 2, 1> MatmulSmall;
typedef MatmulShape<2, 2, 2, 2, 2> MatmulSplit2;
typedef MatmulShape<2, 2, 2, 2, 4> MatmulSplit4;

// Which large tile: 256 x 256 (4), 256 x 192 (3), or neither (0). One
// workgroup fills a CU, so the time is the rounds it takes over the CUs times
// a round's. In units of a 128-block on 16 columns per wave (0.4 us) a round
// of 64 tn columns takes tn KB and 20 for its beginning and end, and one of
// two 128 x 128 tiles per CU 2.7 KB and 14 (measured at 8192 x 8192 x 8192,
// 32768 x 16384 x 4096 and 4096 x 6144 x 2048).
int large_tile(const MatmulArgs& p) {
  const long long tm = ceil_div(p.M, 256);
  const double kb = p.KB;
  const double mid = ceil_div(ceil_div(p.M, 128) * ceil_div(p.N, 128), 2 * kCUs) * (2.7 * kb + 14.0);
  const double l4 = ceil_div(tm * ceil_div(p.N, 256), kCUs) * (4.0 * kb + 20.0);
  const double l3 = ceil_div(tm * ceil_div(p.N, 192), kCUs) * (3.0 * kb + 20.0);
  if (mid < l4 && mid < l3) return 0;
  return l4 <= l3 ? 4 : 3;
}

template <class S, int MODE, bool E8, int ROWS, bool F32OUT>
int launch_matmul(const MatmulArgs& p, bool direct, hipStream_t s) {
  const long long grid = ceil_div(p.M, S::BM) * ceil_div(p.N, S::BN);
  return direct ? launch(matmul_kernel<S, MODE, E8, ROWS, F32OUT, true>, grid, S::NT * S::KS, s, p)
                : launch(matmul_kernel<S, MODE, E8, ROWS, F32OUT, false>, grid, S::NT * S::KS, s, p);
}
template <int MODE, bool E8, int ROWS, bool F32OUT, int MT, int NT, int UN>
int launch_matmul_few(const MatmulArgs& p, hipStream_t s) {
  constexpr int M8 = MODE == kMulE8m0 ? kMulScale : MODE;
  return launch(matmul_few_kernel<M8, E8, ROWS, F32OUT, MT, NT, UN>, ceil_div(p.N, 16 * NT), 512, s, p);
}

template <int MODE, bool E8, int ROWS, bool F32OUT>
int launch_matmul_shape(const MatmulArgs& p, bool direct, hipStream_t s) {
  // Few rows: each workgroup reads all of a, so it takes as many columns as
  // leave a workgroup for most CUs (16 x 12288 x 4096: 11.9 us with 64 columns,
  // 15.0 with 16; 32 x 8192 x 4096: 12.3 with 32, 14.9 with 16, 14.8 with 64).
  // With 33 to 64 rows that is too much to read as soon as the CUs take turns:
  // 64 x 4096 x 4096 takes 11.7 us in tiles (bf16) against 13.3, and fp32
  // results, whose tiles cost twice the instructions, 16.3 against 13.5, but
  // 64 x 8192 x 4096 18.6 against 25.0.
  const long long n16 = ceil_div(p.N, 16);
  if (direct && p.M <= 32) {
    if (n16 >= 3 * kCUs)
      return p.M <= 16 ? launch_matmul_few<MODE, E8, ROWS, F32OUT, 1, 4, 1>(p, s)
                       : launch_matmul_few<MODE, E8, ROWS, F32OUT, 2, 4, 1>(p, s);
    if (n16 >= 2 * kCUs)
      return p.M <= 16 ? launch_matmul_few<MODE, E8, ROWS, F32OUT, 1, 2, 2>(p, s)
                       : launch_matmul_few<MODE, E8, ROWS, F32OUT, 2, 2, 2>(p, s);
    return p.M <= 16 ? launch_matmul_few<MODE, E8, ROWS, F32OUT, 1, 1, 4>(p, s)
                     : launch_matmul_few<MODE, E8, ROWS, F32OUT, 2, 1, 2>(p, s);
  }
  if (direct && p.M <= 64 && n16 <= (F32OUT ? kCUs : kCUs / 2))
    return launch_matmul_few<MODE, E8, ROWS, F32OUT, 4, 1, 2>(p, s);
  if constexpr (MODE != kMulExact) {
    const int tn = direct ? large_tile(p) : 0;
    if (tn == 4)
      return launch(matmul_large_kernel<4, MODE, E8, ROWS>, ceil_div(p.M, 256) * ceil_div(p.N, 256), 512, s, p);
    if (tn == 3)
      return launch(matmul_large_kernel<3, MODE, E8, ROWS>, ceil_div(p.M, 256) * ceil_div(p.N, 192), 512, s, p);
  }
  if (ceil_div(p.M, 128) * ceil_div(p.N, 128) >= kCUs)
    return launch_matmul<MatmulMid, MODE, E8, ROWS, F32OUT>(p, direct, s);
  // too few tiles for every CU: what counts is the number of steps, each as
  // long as its loads take. 256 x 4096 x 4096 takes 18.5 us in one group of
  // waves, 14.2 in two, 12.4 in four; where the loads go through registers
  // four groups run short of them (777 x 1000 x 1333, fp32: 16.4, 14.7, 24.5)
  if (ceil_div(p.M, 64) * ceil_div(p.N, 64) <= kCUs && p.KB >= 4)
    return direct ? launch(matmul_kernel<MatmulSplit4, MODE, E8, ROWS, F32OUT, true>,
                           ceil_div(p.M, 64) * ceil_div(p.N, 64), 1024, s, p)
                  : launch(matmul_kernel<MatmulSplit2, MODE, E8, ROWS, F32OUT, false>,
                           ceil_div(p.M, 64) * ceil_div(p.N, 64), 512, s, p);
  return launch_matmul<MatmulSmall, MODE, E8, ROWS, F32OUT>(p, direct, s);
}
template <int MODE, bool E8, bool F32OUT>
int launch_matmul_rows(const MatmulArgs& p, int rows, bool direct, hipStream_t s) {
  return rows == 1 ? launch_matmul_shape<MODE, E8, 1, F32OUT>(p, direct, s)
                   : launch_matmul_shape<MODE, E8, 128, F32OUT>(p, direct, s);
}

}  // namespace
}  // namespace pararnn

using namespace pararnn;

extern "C" int32_t pararnn_gated_workspace_bytes(int32_t adjoint, const pararnn_gated_opts* o, size_t* bytes) {
  if ((adjoint != 0 && adjoint != 1) || !bytes || !gated_ok(o, adjoint != 0)) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  size_t n = 0;
  for (int C = 1; C <= kScanMaxC; C *= 2) {
    if (o->D % C) continue;
    const size_t t = gated_layout(o, adjoint != 0, C).total;
    n = t > n ? t : n;
  }
  *bytes = n;
  return PARARNN_OK;
}

extern "C" int32_t pararnn_gated_saved_rows(int32_t L) {
  return L < 1 ? 0 : static_cast<int32_t>(ceil_div(L, kGatedSave));
}

extern "C" int32_t pararnn_gated_scan(const void* u, const float* lam, const float* h0, void* h, float* hT,
                                      float* saved, void* ws, size_t ws_bytes, const pararnn_gated_opts* o,
                                      void* stream) {
  if (!gated_ok(o, false) || !u || !lam || !h) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = o->dtype == PARARNN_BF16 ? 2 : 4;
  const int C = pick_c(kScanMaxC, o->D, es, {u, h}, {hT, saved});
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
  if (!gated_ok(o, true) || !u || !lam || !saved || !dh || !du) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = o->dtype == PARARNN_BF16 ? 2 : 4;
  const int C = pick_c(kScanMaxC, o->D, es, {u, dh, du}, {saved, dh0});
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

extern "C" int32_t pararnn_norm_residual(const void* x, const void* residual, const float* w, void* s, void* y,
                                         void* scale, const pararnn_norm_opts* o, void* stream_) {
  if (!norm_ok(o) || !x || !w || !y) return PARARNN_EINVAL;
  if (o->out < PARARNN_NORM_SAME || o->out > PARARNN_NORM_FP8_E8M0) return PARARNN_EINVAL;
  if (o->out != PARARNN_NORM_SAME && !scale) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = o->dtype == PARARNN_BF16 ? 2 : 4;
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(s, es) || !aligned(w, 4) ||
      (o->out == PARARNN_NORM_SAME && !aligned(y, es)) || (o->out == PARARNN_NORM_FP8 && !aligned(scale, 4)))
    return PARARNN_EUNSUPPORTED;
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.residual = residual;
  a.w = w;
  a.s = s;
  a.y = y;
  a.scale = scale;
  a.N = o->N;
  a.D = o->D;
  a.eps = o->eps;
  const bool stream = norm_stream(o, static_cast<int>(es) * 3 + 1);
  hipStream_t st = static_cast<hipStream_t>(stream_);
  const bool vec = norm_vec(o->D, {x, residual, w, s, y});
  if (o->dtype == PARARNN_BF16)
    return vec ? launch_norm_out<bf16, true>(o->out, a, stream, st) : launch_norm_out<bf16, false>(o->out, a, stream, st);
  return vec ? launch_norm_out<float, true>(o->out, a, stream, st) : launch_norm_out<float, false>(o->out, a, stream, st);
}

extern "C" size_t pararnn_norm_workspace_bytes(const pararnn_norm_opts* o) {
  if (!norm_ok(o) || !dtype_ok(o->dtype)) return 0;
  return round_up(sizeof(float) * static_cast<size_t>(norm_adjoint_grid(o)) * o->D);
}

extern "C" int32_t pararnn_norm_residual_adjoint(const void* s, const float* w, const void* dy, const void* ds,
                                                 void* dx, float* dw, void* ws, size_t ws_bytes,
                                                 const pararnn_norm_opts* o, void* stream_) {
  if (!norm_ok(o) || !s || !w || !dy || !dx || (dw && !ws)) return PARARNN_EINVAL;
  if (!dtype_ok(o->dtype)) return PARARNN_EUNSUPPORTED;
  const size_t es = o->dtype == PARARNN_BF16 ? 2 : 4;
  if (!aligned(s, es) || !aligned(dy, es) || !aligned(ds, es) || !aligned(dx, es) || !aligned(w, 4) || !aligned(dw, 4))
    return PARARNN_EUNSUPPORTED;
  if (dw && ws_bytes < pararnn_norm_workspace_bytes(o)) return PARARNN_EWORKSPACE;
  if (dw && !aligned(ws, kAlign)) return PARARNN_EUNSUPPORTED;
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = s;
  a.w = w;
  a.dy = dy;
  a.ds = ds;
  a.dx = dx;
  a.dw_part = dw ? static_cast<float*>(ws) : nullptr;
  a.N = o->N;
  a.D = o->D;
  a.eps = o->eps;
  const bool stream = norm_stream(o, static_cast<int>(es) * 4);
  hipStream_t st = static_cast<hipStream_t>(stream_);
  const bool vec = norm_vec(o->D, {s, w, dy, ds, dx});
  const long long grid = norm_adjoint_grid(o);
  int rc;
  if (o->dtype == PARARNN_BF16)
    rc = vec ? launch_norm_adjoint<bf16, true>(a, grid, stream, st) : launch_norm_adjoint<bf16, false>(a, grid, stream, st);
  else
    rc = vec ? launch_norm_adjoint<float, true>(a, grid, stream, st) : launch_norm_adjoint<float, false>(a, grid, stream, st);
  if (rc || !dw) return rc;
  return launch(column_sum_kernel, ceil_div(o->D, kSumCols), kSumCols * kSumGroups, st,
                static_cast<const float*>(a.dw_part), dw, grid, static_cast<int>(o->D),
                static_cast<const float*>(nullptr), 0.0f);
}

extern "C" int32_t pararnn_matmul_fp8(const void* a, const void* sa, const void* w, const void* sw, const float* bias,
                                      void* y, const pararnn_matmul_opts* o, void* stream_) {
  if (!o || o->M < 1 || o->N < 1 || o->K < 1 || !a || !sa || !w || !sw || !y) return PARARNN_EINVAL;
  if (o->w_rows != 1 && o->w_rows != 128) return PARARNN_EINVAL;
  if (o->scale != PARARNN_SCALE_F32 && o->scale != PARARNN_SCALE_E8M0) return PARARNN_EINVAL;
  if (!dtype_ok(o->y_dtype)) return PARARNN_EUNSUPPORTED;
  const bool e8 = o->scale == PARARNN_SCALE_E8M0, f32 = o->y_dtype == PARARNN_F32;
  if (!aligned(bias, 4) || !aligned(y, f32 ? 4 : 2) || (!e8 && (!aligned(sa, 4) || !aligned(sw, 4))))
    return PARARNN_EUNSUPPORTED;
  if (o->M > 2147483647 - 256 || o->N > 2147483647 - 256 || o->K > (1 << 22)) return PARARNN_EINVAL;
  if (static_cast<double>(ceil_div(o->M, 64)) * ceil_div(o->N, 64) > 2.0e9) return PARARNN_EINVAL;
  MatmulArgs p;
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
  p.stream = 2.0 * p.M * p.N > 256.0 * 1024 * 1024;
  const bool direct = o->K % 16 == 0 && aligned(a, 16) && aligned(w, 16);
  hipStream_t s = static_cast<hipStream_t>(stream_);
  const int rows = o->w_rows;
  if (f32) return e8 ? launch_matmul_rows<kMulExact, true, true>(p, rows, direct, s)
                     : launch_matmul_rows<kMulExact, false, true>(p, rows, direct, s);
  return e8 ? launch_matmul_rows<kMulE8m0, true, false>(p, rows, direct, s)
            : launch_matmul_rows<kMulScale, false, false>(p, rows, direct, s);
}
