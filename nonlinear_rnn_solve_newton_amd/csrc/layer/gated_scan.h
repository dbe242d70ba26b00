// gated_scan.h -- gated linear recurrence over a sequence, its adjoint and its
// single-token step. Per channel d, with gate inputs u = (u_r, u_i, x) and
// r = s(u_r), i = s(u_i) (s: logistic sigmoid):
//   log a_t = -c softplus(lam) r_t,   a_t = exp(log a_t) in (0, 1],
//   m_t = sqrt(1 - a_t^2),            h_t = a_t h_{t-1} + m_t i_t x_t.
// A document start (reset) counts h_{t-1} as zero; a step at or past the row's
// length leaves the state as it is and puts out zero.
//
// Adjoint for g_t = dL/dh_t, on mu_t = a_t (mu_{t+1} + dh_t) (the gradient that
// step t passes back; mu past the end is dL/dhT):
//   g_t = mu_{t+1} + dh_t,   du_x = g m i,   du_i = g m x i (1 - i),
//   dlog a = g a (h_{t-1} - i x a / m),   du_r = dlog a (-c softplus(lam)) r (1 - r),
//   dlam = -c s(lam) sum_t dlog a r,      dL/dh0 = mu_0.
//
// Both are linear scans, bound by HBM: bf16 moves 8 bytes per element forward
// (u in, h out) and 14 back (u and dh in, du out). The states between the
// chunks of 96 steps (4 / 96 bytes per element) are what the forward pass
// leaves for the adjoint, which rebuilds the others from u, in 32 bits: less
// to move than the states themselves, and not rounded to bf16.
//
// Measured, bf16: 8 x 4096 x 1024 takes 60.5 us forward (268 MB, 4.4 TB/s) and
// 110 us back (470 MB, 4.3 TB/s), 1 x 65536 x 2048 takes 213 us forward (5.0
// TB/s), against 5.5 TB/s that a plain stream of that mix reaches. Between them
// lie the arithmetic (34 vector instructions per element forward, 65 back: half
// of the issue slots, and a fifth more as the transcendental ones take two), the
// launch that clears the carries (5 us) and, where few chunks are in flight,
// the wait for the carry (2 us per group of chunks).
#pragma once

#include <type_traits>

#include "layer_common.h"

namespace pararnn {

constexpr int kGatedSave = 96;  // steps between two saved states: an adjoint chunk

// n / d for n < 2^31 by a multiplication: m = ceil(2^(31 + s) / d), s = ceil(log2 d)
struct FastDiv {
  uint32_t m, s;
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> (31 + s));
  }
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return FastDiv{static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d), s};
}

struct GatedArgs {
  const void* u;            // [B][L][3][D]
  const float* lam;         // [D]
  const float* h0;          // [B][D] or nullptr (zero)
  const int* lengths;       // [B] or nullptr (L)
  const unsigned char* reset;  // [B][L] or nullptr
  void* h;                  // [B][L][D]
  float* hT;                // [B][D] or nullptr
  float* saved;             // [ceil(L / kGatedSave)][B][D]; nullptr: none (forward)
  const void* dh;           // [B][L][D]
  const float* dhT;         // [B][D] or nullptr (zero)
  void* du;                 // [B][L][3][D]
  float* dh0;               // [B][D] or nullptr
  float* dl_part;           // [nchunks][B][D] partial sums of dlog a r, or nullptr
  float* dlam;              // [D], where there is one partial sum per channel
  unsigned long long* carry;  // [ngroups][slots] states at the groups' starts
  unsigned long long* agg;    // [nchunks][2][slots] chunk transforms
  unsigned int* ctr;        // ticket counters
  int parts_log2;           // how many of them
  unsigned int run;         // tiles per counter
  FastDiv by_run, by_row;   // division by run and by ntiles_d
  int B, L, D, nchunks, ntiles_d, group;
  float c;
};

// Gate values of one step; y = log2 a = beta2 r with beta2 = -c softplus(lam) log2(e).
// v = 1 - a^2 = 1 - 2^(2y): where it is under 0.22 (2y ln 2 > -0.25) by y q(y), q of
// degree 4 through the Chebyshev points (relative error 1.2e-8), since the
// subtraction would cancel its digits; above, the cancellation costs 2 bits.
struct GateVal {
  float r, i, a, v;
};
__device__ __forceinline__ GateVal gate_values(float ur, float ui, float beta2) {
  GateVal g;
  g.r = sigm(ur);
  g.i = sigm(ui);
  const float y = beta2 * g.r;
  g.a = __builtin_amdgcn_exp2f(y);
  float q = -0.0384703129529953f;
  q = fmaf(q, y, -0.15323998034000397f);
  q = fmaf(q, y, -0.44399136304855347f);
  q = fmaf(q, y, -0.9609050750732422f);
  q = fmaf(q, y, -1.3862943649291992f);
  g.v = y > -0.18033688f ? q * y : fmaf(-g.a, g.a, 1.0f);
  return g;
}
constexpr float kNoInput = 9.0e18f;  // 1/m from here on: m = 0
__device__ __forceinline__ float decay_log2(float lam, float c) { return -1.4426950408889634f * c * softplus(lam); }

// Affine transforms x -> A x + b of C channels. RST: a transform that begins a
// document (anywhere inside) holds A = -0 and drops what comes before it
// altogether, so that an infinity or a NaN of one document does not reach the
// next as 0 x inf. Decays are +0 or more, and a product of them keeps a -0
// factor's sign.
constexpr uint32_t kResetA = 0x80000000u;
template <int C, bool RST>
struct Lin {
  float A[C], b[C];

  __device__ __forceinline__ void set_identity() {
#pragma unroll
    for (int c = 0; c < C; ++c) { A[c] = 1.0f; b[c] = 0.0f; }
  }
  // this <- this o e (e first)
  __device__ __forceinline__ void after(const Lin& e) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float nb = fmaf(A[c], e.b[c], b[c]), nA = A[c] * e.A[c];
      if constexpr (RST) {
        const bool cut = __float_as_uint(A[c]) == kResetA;
        b[c] = cut ? b[c] : nb;
        A[c] = cut ? A[c] : nA;
      } else {
        b[c] = nb;
        A[c] = nA;
      }
    }
  }
  __device__ __forceinline__ void apply(float (&x)[C]) const {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float y = fmaf(A[c], x[c], b[c]);
      x[c] = (RST && __float_as_uint(A[c]) == kResetA) ? b[c] : y;
    }
  }
  __device__ __forceinline__ Lin shfl_down(int delta) const {
    Lin r;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      r.A[c] = __shfl_down(A[c], delta, 64);
      r.b[c] = __shfl_down(b[c], delta, 64);
    }
    return r;
  }
  __device__ __forceinline__ Lin shfl_up(int delta) const {
    Lin r;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      r.A[c] = __shfl_up(A[c], delta, 64);
      r.b[c] = __shfl_up(b[c], delta, 64);
    }
    return r;
  }
};

// The document starts among a lane's T steps, bit t for step t. The wave's
// steps begin at l and are read a byte per lane; a step at or past len is none.
template <int T, int LL, bool RST>
__device__ __forceinline__ uint32_t document_starts(const GatedArgs& p, int b, int l, int len, int lane) {
  static_assert(T <= 32 && T * LL <= 64, "a byte per lane");
  if constexpr (RST) {
    const bool in = lane < T * LL && l + lane < len;
    const unsigned char v = in ? p.reset[static_cast<long long>(b) * p.L + l + lane] : 0;
    const unsigned long long all = __ballot(v != 0);
    return static_cast<uint32_t>(all >> (lane / (64 / LL) * T)) & static_cast<uint32_t>((1ull << T) - 1);
  }
  return 0u;
}
template <bool RST>
__device__ __forceinline__ float marked(float a, uint32_t cuts, int t) {
  return RST && (cuts >> t & 1u) ? __uint_as_float(kResetA) : a;
}

// Which tile (batch row, channels) and chunk a workgroup works on. The tiles
// are dealt out in `parts` equal runs, each with a ticket counter of its own (a
// counter that 512 workgroups ask at once costs the last of them 3 us); within
// a run the tickets go chunk by chunk. Workgroup i takes a ticket of run
// i % parts (the last run may be short: its spare tickets are of no tile).
// Chunks of a tile depend on earlier ones of that tile only, so whatever a
// workgroup waits for has started before it. A run is neighbouring tiles; with
// lengths every parts-th one, since workgroups go to the XCDs in turn and a run
// of short rows would leave its XCDs idle (8 rows of up to 3000 steps x 512: 35
// -> 29 us forward, 55 -> 44 us back).
struct TilePos {
  int chunk, tile, b, dt0;
};
constexpr int kTicketStride = 64;  // counters 256 bytes apart
struct Tickets {
  unsigned int part;
  __device__ __forceinline__ explicit Tickets(const GatedArgs& p) { part = blockIdx.x & ((1u << p.parts_log2) - 1u); }
  // by one thread; with one chunk nothing waits, and the order is that of the workgroups
  __device__ __forceinline__ unsigned int take(const GatedArgs& p) const {
    return p.nchunks > 1 ? atomicAdd(p.ctr + part * kTicketStride, 1u) : blockIdx.x >> p.parts_log2;
  }
  __device__ __forceinline__ bool fill(const GatedArgs& p, unsigned int chunk, unsigned int tile, int cw, TilePos* at) const {
    at->chunk = static_cast<int>(chunk);
    at->tile = static_cast<int>(tile);
    at->b = static_cast<int>(p.by_row.div(tile));
    at->dt0 = static_cast<int>(tile - static_cast<unsigned int>(at->b) * p.ntiles_d) * cw;
    return tile < static_cast<unsigned int>(p.B) * p.ntiles_d;
  }
  // one chunk: workgroup i has tile i
  __device__ __forceinline__ void one(const GatedArgs& p, unsigned int i, int cw, TilePos* at) const {
    fill(p, 0u, i, cw, at);
  }
  __device__ __forceinline__ bool place(const GatedArgs& p, unsigned int ticket, int cw, TilePos* at) const {
    const unsigned int chunk = p.by_run.div(ticket);
    const unsigned int k = ticket - chunk * p.run;
    return fill(p, chunk, p.lengths ? (k << p.parts_log2) + part : part * p.run + k, cw, at);
  }
};

// Parked values are read back, not kept in registers after all: volatile
__device__ __forceinline__ f32x4 read_back(const f32x4* p) {
  return *(const volatile __attribute__((address_space(3))) f32x4*)p;
}

// The carry into a chunk. Chunks (counted in scan order) form groups of
// `group` <= kMaxGroup. A chunk publishes its own transform as soon as it has
// it, except the last of a group, which publishes the state at its end: the
// next group's start. A chunk so waits for its group's start and for the
// transforms of the chunks before it in the group, reads them all at once and
// composes them in order: the chain of waits has one link per group, not per
// chunk, and the order of the sums does not depend on timing, so results
// repeat bit for bit. Tickets are taken chunk by chunk, so whatever a
// workgroup waits for has started before it. Words carry their tag (1:
// written) in the high half. Called by one wave, a channel per lane: tot is
// the chunk's transform, x the state before the first chunk; returns the
// state before chunk q.
constexpr int kMaxGroup = 8;
template <bool RST>
__device__ __forceinline__ float chunk_carry(const GatedArgs& p, long long slots, long long chan, int q,
                                             const Lin<1, RST>& tot, float x) {
  const int grp = q / p.group, j = q - grp * p.group;
  const bool last = j == p.group - 1;
  if (!last && q < p.nchunks - 1) {
    desc_put(p.agg + static_cast<long long>(q) * 2 * slots + chan, 1u, tot.A[0]);
    desc_put(p.agg + (static_cast<long long>(q) * 2 + 1) * slots + chan, 1u, tot.b[0]);
  }
  unsigned long long wa[kMaxGroup - 1], wb[kMaxGroup - 1], wx = 0ull;
  while (true) {
    const unsigned long long* at = p.agg + static_cast<long long>(q - j) * 2 * slots + chan;
#pragma unroll
    for (int s = 0; s < kMaxGroup - 1; ++s) {
      if (s < j) {
        wa[s] = desc_get(const_cast<unsigned long long*>(at) + 2 * s * slots);
        wb[s] = desc_get(const_cast<unsigned long long*>(at) + (2 * s + 1) * slots);
      }
    }
    if (grp > 0) wx = desc_get(p.carry + static_cast<long long>(grp) * slots + chan);
    bool ok = grp == 0 || desc_ok(wx, 1u);
#pragma unroll
    for (int s = 0; s < kMaxGroup - 1; ++s)
      if (s < j) ok = ok && desc_ok(wa[s], 1u) && desc_ok(wb[s], 1u);
    if (ok) break;
    __builtin_amdgcn_s_sleep(1);
  }
  float v[1] = {grp > 0 ? desc_val(wx) : x};
#pragma unroll
  for (int s = 0; s < kMaxGroup - 1; ++s) {
    if (s < j) {
      Lin<1, RST> e;
      e.A[0] = desc_val(wa[s]);
      e.b[0] = desc_val(wb[s]);
      e.apply(v);
    }
  }
  if (last && q < p.nchunks - 1) {
    float y[1] = {v[0]};
    tot.apply(y);
    desc_put(p.carry + static_cast<long long>(grp + 1) * slots + chan, 1u, y[0]);
  }
  return v[0];
}

// Chunks of a row that hold steps of it; at least one, which passes the state
// on. Later ones only put out zeros: they load nothing and nobody waits for
// them (16 rows of up to 2048 steps, 41% of them live, 1024 channels: 69 -> 54
// us forward, 127 -> 93 us back).
template <int CL>
__device__ __forceinline__ int live_chunks(int len) {
  return max((len + CL - 1) / CL, 1);
}

// A workgroup covers LD * C channels (LD = 64 / LL lanes along D) and
// CL = W * LL * T steps: T steps in series per lane, a shuffle scan over the
// LL lane groups, an LDS scan over the W waves, chunk_carry over the chunks.
// ONE: the whole sequence is one chunk (no ticket, no carry).
// The first wave takes the carry. It parks its steps in workgroup memory
// meanwhile: the words it polls would otherwise cost every wave registers.
template <class UT, int C, int T, int W, int LL, int OCC, bool RST, bool ONE>
__global__ void __launch_bounds__(64 * W, OCC) gated_scan_kernel(const GatedArgs p) {
  constexpr int LD = 64 / LL, CW = LD * C, CL = W * LL * T;
  static_assert(CW <= 64, "one wave takes the carry, a channel per lane");
  constexpr int NP = 2 * T * C / 4;  // 16-byte pieces that a lane parks
  static_assert(T * C % 4 == 0, "whole pieces");
  __shared__ float s_A[W][CW], s_b[W][CW], s_start[W][CW], s_beta[CW];
  __shared__ f32x4 s_park[ONE ? 1 : NP][64];
  __shared__ unsigned int s_ticket;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Tickets q(p);
  TilePos at;
  if constexpr (ONE) {
    q.one(p, blockIdx.x, CW, &at);
  } else {
    if (tid == 0) s_ticket = q.take(p);
    __syncthreads();
    if (!q.place(p, __builtin_amdgcn_readfirstlane(s_ticket), CW, &at)) return;
  }
  const int chunk = at.chunk, tile = at.tile, b = at.b, dt0 = at.dt0;

  const int ld = lane % LD, ll = lane / LD;
  const int d0 = dt0 + ld * C;
  const bool dv = d0 < p.D;
  const int lt0 = (wave * LL + ll) * T;
  const int l0 = chunk * CL + lt0;
  const int len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
  const long long wrow = static_cast<long long>(b) * p.L + static_cast<long long>(chunk) * CL;
  const uint32_t gstep = static_cast<uint32_t>(p.D * sizeof(UT)), ustep = 3 * gstep;
  const uint32_t rows = static_cast<uint32_t>(min(p.L - chunk * CL, CL));
  constexpr uint32_t kOOB = 0x80000000u;  // extents stay below 2^31 bytes
  const uint32_t vd = static_cast<uint32_t>(d0 * sizeof(UT));
  const uint32_t vu0 = dv ? static_cast<uint32_t>(lt0) * ustep + vd : kOOB;
  const uint32_t vh0 = dv ? static_cast<uint32_t>(lt0) * gstep + vd : kOOB;
  const __amdgpu_buffer_rsrc_t ru = make_rsrc(static_cast<const UT*>(p.u) + wrow * 3 * p.D, rows * ustep);
  const __amdgpu_buffer_rsrc_t rh = make_rsrc(static_cast<UT*>(p.h) + wrow * p.D, rows * gstep);

  const int last = live_chunks<CL>(len) - 1;
  if constexpr (!ONE) {
    if (chunk > last) {
      const float zero[C] = {};
#pragma unroll
      for (int t = 0; t < T; ++t) buf_st<UT, C>(rh, vh0 + t * gstep, 0u, zero);
      return;
    }
  }
  URaw<UT, C> uu[T][3];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int g = 0; g < 3; ++g) uu[t][g].load(ru, vu0 + t * ustep, static_cast<uint32_t>(g) * gstep);
  const uint32_t cuts = document_starts<T, LL, RST>(p, b, chunk * CL + wave * LL * T, len, lane);
  if (tid < CW) s_beta[tid] = decay_log2(p.lam[min(dt0 + tid, p.D - 1)], p.c);
  __syncthreads();
  float beta2[C];
#pragma unroll
  for (int c = 0; c < C; ++c) beta2[c] = s_beta[ld * C + c];

  // the steps' transforms; those past the length are the identity
  const bool ragged = (chunk + 1) * static_cast<long long>(CL) > len;
  float A[T][C], x[T][C];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const GateVal g = gate_values(uu[t][0].get(c), uu[t][1].get(c), beta2[c]);
      A[t][c] = g.a;
      x[t][c] = __builtin_amdgcn_sqrtf(g.v) * (g.i * uu[t][2].get(c));
    }
  if (ragged) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        A[t][c] = l0 + t < len ? A[t][c] : 1.0f;
        x[t][c] = l0 + t < len ? x[t][c] : 0.0f;
      }
  }

  // the lane's steps, then the lane groups of the wave
  Lin<C, RST> acc;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    Lin<C, RST> e;
#pragma unroll
    for (int c = 0; c < C; ++c) { e.A[c] = marked<RST>(A[t][c], cuts, t); e.b[c] = x[t][c]; }
    if (t) e.after(acc);
    acc = e;
  }
  Lin<C, RST> excl;
  excl.set_identity();
  if constexpr (LL > 1) {
#pragma unroll
    for (int off = 1; off < LL; off *= 2) {
      const Lin<C, RST> prev = acc.shfl_up(off * LD);
      if (ll >= off) acc.after(prev);
    }
    const Lin<C, RST> prev = acc.shfl_up(LD);
    if (ll > 0) excl = prev;
  }
  if (ll == LL - 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s_A[wave][ld * C + c] = acc.A[c];
      s_b[wave][ld * C + c] = acc.b[c];
    }
  }
  __syncthreads();
  if (wave == 0) {
    float* flat_A = &A[0][0];
    float* flat_x = &x[0][0];
#pragma unroll
    for (int i = 0; i < (ONE ? 0 : NP / 2); ++i) {
      s_park[i][lane] = f32x4{flat_A[4 * i], flat_A[4 * i + 1], flat_A[4 * i + 2], flat_A[4 * i + 3]};
      s_park[NP / 2 + i][lane] = f32x4{flat_x[4 * i], flat_x[4 * i + 1], flat_x[4 * i + 2], flat_x[4 * i + 3]};
    }
    if (lane < CW) {
      const bool in = dt0 + lane < p.D;
      const long long bd = static_cast<long long>(b) * p.D + dt0 + lane;
      float v[1] = {in && p.h0 ? p.h0[bd] : 0.0f};
      if constexpr (!ONE) {
        Lin<1, RST> tot;
        tot.set_identity();
#pragma unroll
        for (int w = 0; w < W; ++w) {
          Lin<1, RST> e;
          e.A[0] = s_A[w][lane];
          e.b[0] = s_b[w][lane];
          e.after(tot);
          tot = e;
        }
        v[0] = chunk_carry<RST>(p, static_cast<long long>(p.B) * p.ntiles_d * CW,
                                static_cast<long long>(tile) * CW + lane, chunk, tot, v[0]);
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        s_start[w][lane] = v[0];
        Lin<1, RST> e;
        e.A[0] = s_A[w][lane];
        e.b[0] = s_b[w][lane];
        e.apply(v);
      }
      if (p.hT && in && (ONE || chunk == last)) p.hT[bd] = v[0];
    }
#pragma unroll
    for (int i = 0; i < (ONE ? 0 : NP / 2); ++i) {
      const f32x4 va = read_back(&s_park[i][lane]), vx = read_back(&s_park[NP / 2 + i][lane]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        flat_A[4 * i + k] = va[k];
        flat_x[4 * i + k] = vx[k];
      }
    }
  }
  __syncthreads();
  float h[C];
#pragma unroll
  for (int c = 0; c < C; ++c) h[c] = s_start[wave][ld * C + c];
  if constexpr (LL > 1) excl.apply(h);
  if (p.saved && dv && l0 % kGatedSave == 0 && l0 < p.L)
    st_f32<C>(p.saved + (static_cast<long long>(l0 / kGatedSave) * p.B + b) * p.D + d0, h);

  auto put_out = [&](auto full) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      Lin<C, RST> e;
#pragma unroll
      for (int c = 0; c < C; ++c) { e.A[c] = marked<RST>(A[t][c], cuts, t); e.b[c] = x[t][c]; }
      e.apply(h);
      float o[C];
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = (!decltype(full)::value && l0 + t >= len) ? 0.0f : h[c];
      buf_st<UT, C>(rh, vh0 + t * gstep, 0u, o);  // dropped past L or D
    }
  };
  if (ragged) put_out(std::false_type{});
  else put_out(std::true_type{});
}

// Packed values stay packed: without this the compiler keeps the unpacked ones
// of their first use in registers for the second.
template <int C>
__device__ __forceinline__ void keep_packed(URaw<bf16, C>& u) {
#pragma unroll
  for (int i = 0; i < URaw<bf16, C>::NW; ++i) __asm__ volatile("" : "+v"(u.w[i]));
}
template <int C>
__device__ __forceinline__ void keep_packed(URaw<float, C>&) {}

// The adjoint of one chunk of CL = kGatedSave steps: a scan forward from the
// saved state for the h_{t-1}, and the scan backward for mu, on the same
// lanes.
template <class UT, int C, int T, int W, int LL, int OCC, bool RST, bool ONE>
__global__ void __launch_bounds__(64 * W, OCC) gated_adjoint_kernel(const GatedArgs p) {
  constexpr int LD = 64 / LL, CW = LD * C, CL = W * LL * T, NSEG = W * LL;
  static_assert(ONE || CL == kGatedSave, "a chunk starts at a saved state");
  static_assert(CW <= 64, "one wave takes the carry, a channel per lane");
  // transforms of the waves, forward (A, b) and backward (B, m); what enters them
  __shared__ float s_A[W][CW], s_b[W][CW], s_B[W][CW], s_m[W][CW], s_h[W][CW], s_mu[W][CW], s_beta[CW];
  __shared__ float s_dl[NSEG][CW];
  constexpr int NP = 5 * T * C / 4;  // 16-byte pieces that a lane of the first wave parks
  static_assert(T * C % 4 == 0, "whole pieces");
  __shared__ f32x4 s_park[ONE ? 1 : NP][64];
  __shared__ Lin<C, RST> s_fx[W][LL > 1 ? 64 : 1], s_bx[W][LL > 1 ? 64 : 1];
  __shared__ unsigned int s_ticket;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ld = lane % LD, ll = lane / LD;
  const int lt0 = (wave * LL + ll) * T;
  const uint32_t gstep = static_cast<uint32_t>(p.D * sizeof(UT)), ustep = 3 * gstep;
  constexpr uint32_t kOOB = 0x80000000u;

  Tickets q(p);
  TilePos at;
  if constexpr (ONE) {
    q.one(p, blockIdx.x, CW, &at);
  } else {
    if (tid == 0) s_ticket = q.take(p);
    __syncthreads();
    if (!q.place(p, __builtin_amdgcn_readfirstlane(s_ticket), CW, &at)) return;
  }
  const int chunk = p.nchunks - 1 - at.chunk;  // taken from the end of L
  const int tile = at.tile, b = at.b, dt0 = at.dt0, d0 = dt0 + ld * C;
  const bool dv = d0 < p.D;
  const int l0 = chunk * CL + lt0;
  const int len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
  const long long wrow = static_cast<long long>(b) * p.L + static_cast<long long>(chunk) * CL;
  const uint32_t rows = static_cast<uint32_t>(min(p.L - chunk * CL, CL));
  const uint32_t vd = static_cast<uint32_t>(d0 * sizeof(UT));
  const uint32_t vu0 = dv ? static_cast<uint32_t>(lt0) * ustep + vd : kOOB;
  const uint32_t vh0 = dv ? static_cast<uint32_t>(lt0) * gstep + vd : kOOB;
  const __amdgpu_buffer_rsrc_t ru = make_rsrc(static_cast<const UT*>(p.u) + wrow * 3 * p.D, rows * ustep);
  const __amdgpu_buffer_rsrc_t rdh = make_rsrc(static_cast<const UT*>(p.dh) + wrow * p.D, rows * gstep);
  const __amdgpu_buffer_rsrc_t rdu = make_rsrc(static_cast<UT*>(p.du) + wrow * 3 * p.D, rows * ustep);

  const int live = live_chunks<CL>(len);
  if constexpr (!ONE) {
    if (chunk >= live) {
      const float zero[C] = {};
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int g = 0; g < 3; ++g) buf_st<UT, C>(rdu, vu0 + t * ustep, static_cast<uint32_t>(g) * gstep, zero);
      if (p.dl_part && tid < CW && dt0 + tid < p.D)
        p.dl_part[(static_cast<long long>(chunk) * p.B + b) * p.D + dt0 + tid] = 0.0f;
      return;
    }
  }
  URaw<UT, C> uu[T][3], gg[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
#pragma unroll
    for (int g = 0; g < 3; ++g) uu[t][g].load(ru, vu0 + t * ustep, static_cast<uint32_t>(g) * gstep);
    gg[t].load(rdh, vh0 + t * gstep, 0u);
  }
  const uint32_t cuts = document_starts<T, LL, RST>(p, b, chunk * CL + wave * LL * T, len, lane);
  if (tid < CW) s_beta[tid] = decay_log2(p.lam[min(dt0 + tid, p.D - 1)], p.c);
  __syncthreads();
  float beta2[C];
#pragma unroll
  for (int c = 0; c < C; ++c) beta2[c] = s_beta[ld * C + c];

  const bool ragged = (chunk + 1) * static_cast<long long>(CL) > len;
  // per step: its transform (bb later holds h_{t-1}), r, i and 1/m; x and dh stay packed
  float A[T][C], bb[T][C], gr[T][C], gi[T][C], im[T][C];
  // the steps one after the other: interleaved, their intermediates would not fit the registers
#pragma unroll
  for (int t = 0; t < T; ++t) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const GateVal g = gate_values(uu[t][0].get(c), uu[t][1].get(c), beta2[c]);
      gr[t][c] = g.r;
      gi[t][c] = g.i;
      // 1/m is kept finite (2^63 for v = 0): where v is 0, so are r or beta, and with them what 1/m multiplies.
      // v is +0 or more; as an integer a NaN is larger than every number and stays one
      im[t][c] = __builtin_amdgcn_rsqf(__uint_as_float(max(__float_as_uint(g.v), 0x00800000u)));
      A[t][c] = g.a;
      bb[t][c] = g.v * im[t][c] * (g.i * uu[t][2].get(c));
    }
  }
  if (ragged) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        A[t][c] = l0 + t < len ? A[t][c] : 1.0f;
        bb[t][c] = l0 + t < len ? bb[t][c] : 0.0f;
        if (c == 0 && l0 + t >= len) gg[t].zero();
      }
  }

  // forward over the lane's steps, and backward: mu_t = A_t mu_{t+1} + A_t dh_t
  Lin<C, RST> fw, bw;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    Lin<C, RST> e;
#pragma unroll
    for (int c = 0; c < C; ++c) { e.A[c] = marked<RST>(A[t][c], cuts, t); e.b[c] = bb[t][c]; }
    if (t) e.after(fw);
    fw = e;
  }
#pragma unroll
  for (int t = T - 1; t >= 0; --t) {
    Lin<C, RST> e;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      e.A[c] = marked<RST>(A[t][c], cuts, t);
      e.b[c] = RST && (cuts >> t & 1u) ? 0.0f : A[t][c] * gg[t].get(c);
    }
    if (t < T - 1) e.after(bw);
    bw = e;
  }
  if constexpr (LL > 1) {
#pragma unroll
    for (int off = 1; off < LL; off *= 2) {
      const Lin<C, RST> prev = fw.shfl_up(off * LD);
      if (ll >= off) fw.after(prev);
      const Lin<C, RST> next = bw.shfl_down(off * LD);
      if (ll < LL - off) bw.after(next);
    }
    // what precedes the lane within the wave, in either direction, waits in
    // workgroup memory for the carry: registers are short
    s_fx[wave][lane] = fw;
    s_bx[wave][lane] = bw;
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    keep_packed<C>(uu[t][2]);
    keep_packed<C>(gg[t]);
  }
  if (ll == LL - 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s_A[wave][ld * C + c] = fw.A[c];
      s_b[wave][ld * C + c] = fw.b[c];
    }
  }
  if (ll == 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s_B[wave][ld * C + c] = bw.A[c];
      s_m[wave][ld * C + c] = bw.b[c];
    }
  }
  __syncthreads();
  if (wave == 0) {
    float* const flat[5] = {&A[0][0], &bb[0][0], &gr[0][0], &gi[0][0], &im[0][0]};
    constexpr int N4 = T * C / 4;
#pragma unroll
    for (int k = 0; k < 5; ++k)
#pragma unroll
      for (int i = 0; i < (ONE ? 0 : N4); ++i)
        s_park[k * N4 + i][lane] = f32x4{flat[k][4 * i], flat[k][4 * i + 1], flat[k][4 * i + 2], flat[k][4 * i + 3]};
    if (lane < CW) {
      const bool in = dt0 + lane < p.D;
      const long long bd = static_cast<long long>(b) * p.D + dt0 + lane;
      float h[1] = {in ? p.saved[static_cast<long long>(chunk) * p.B * p.D + bd] : 0.0f};
      float v[1] = {in && p.dhT ? p.dhT[bd] : 0.0f};
      Lin<1, RST> tot;
      tot.set_identity();
#pragma unroll
      for (int w = 0; w < W; ++w) {
        s_h[w][lane] = h[0];
        Lin<1, RST> e;
        e.A[0] = s_A[w][lane];
        e.b[0] = s_b[w][lane];
        e.apply(h);
        e.A[0] = s_B[W - 1 - w][lane];
        e.b[0] = s_m[W - 1 - w][lane];
        e.after(tot);
        tot = e;
      }
      if constexpr (!ONE)
        v[0] = chunk_carry<RST>(p, static_cast<long long>(p.B) * p.ntiles_d * CW,
                                static_cast<long long>(tile) * CW + lane, live - 1 - chunk, tot, v[0]);
#pragma unroll
      for (int w = W - 1; w >= 0; --w) {
        s_mu[w][lane] = v[0];
        Lin<1, RST> e;
        e.A[0] = s_B[w][lane];
        e.b[0] = s_m[w][lane];
        e.apply(v);
      }
    }
#pragma unroll
    for (int k = 0; k < 5; ++k)
#pragma unroll
      for (int i = 0; i < (ONE ? 0 : N4); ++i) {
        const f32x4 v = read_back(&s_park[k * N4 + i][lane]);
#pragma unroll
        for (int q = 0; q < 4; ++q) flat[k][4 * i + q] = v[q];
      }
  }
  __syncthreads();
  float h[C], mu[C], dl[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    h[c] = s_h[wave][ld * C + c];
    mu[c] = s_mu[wave][ld * C + c];
    dl[c] = 0.0f;
  }
  if constexpr (LL > 1) {
    if (ll > 0) s_fx[wave][lane - LD].apply(h);
    if (ll < LL - 1) s_bx[wave][lane + LD].apply(mu);
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    Lin<C, RST> e;
    float prev[C];
#pragma unroll
    for (int c = 0; c < C; ++c) { e.A[c] = marked<RST>(A[t][c], cuts, t); e.b[c] = bb[t][c]; prev[c] = h[c]; }
    e.apply(h);
#pragma unroll
    for (int c = 0; c < C; ++c) bb[t][c] = prev[c];
  }

  auto put_out = [&](auto full) {
#pragma unroll
    for (int t = T - 1; t >= 0; --t) {
      __builtin_amdgcn_sched_barrier(0);
      const bool on = decltype(full)::value || l0 + t < len;
      float o[3][C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const bool ct = RST && (cuts >> t & 1u);
        const float at = A[t][c];
        const float r = gr[t][c], i = gi[t][c], g = mu[c] + gg[t].get(c);
        const float prev = ct ? 0.0f : bb[t][c];
        const float ix = i * uu[t][2].get(c), gx = im[t][c] >= kNoInput ? 0.0f : g * __builtin_amdgcn_rcpf(im[t][c]);
        const float ga = g * at;
        const float dla = ga * fmaf(-ix * at, im[t][c], prev);
        dl[c] = on ? fmaf(dla, r, dl[c]) : dl[c];
        o[0][c] = on ? dla * (0.6931471805599453f * beta2[c]) * fmaf(-r, r, r) : 0.0f;
        o[1][c] = on ? gx * (ix * (1.0f - i)) : 0.0f;
        o[2][c] = on ? gx * i : 0.0f;
        mu[c] = ct ? 0.0f : (on ? ga : mu[c]);
      }
#pragma unroll
      for (int g = 0; g < 3; ++g)
        buf_st<UT, C, kBufNT>(rdu, vu0 + t * ustep, static_cast<uint32_t>(g) * gstep, o[g]);
    }
  };
  if (ragged) put_out(std::false_type{});
  else put_out(std::true_type{});
  // from the lane's steps, each of which adds before it multiplies: the transforms' products, added
  // where mu and dh cancel, would round more
  if (p.dh0 && dv && l0 == 0) st_f32<C>(p.dh0 + static_cast<long long>(b) * p.D + d0, mu);
  if (p.dl_part || p.dlam) {  // the lane groups' sums of dlog a r, added in order
#pragma unroll
    for (int c = 0; c < C; ++c) s_dl[wave * LL + ll][ld * C + c] = dl[c];
    __syncthreads();
    if (wave == 0 && lane < CW && dt0 + lane < p.D) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < NSEG; ++k) v += s_dl[k][lane];
      const int d = dt0 + lane;
      if (p.dlam) p.dlam[d] = -p.c * sigm(p.lam[d]) * v;
      else p.dl_part[(static_cast<long long>(chunk) * p.B + b) * p.D + d] = v;
    }
  }
}

// out[d] = f(d) * sum of `rows` partial rows, in a fixed order: kSumGroups
// interleaved row groups per column, then the groups in turn.
// lam: f = -c s(lam[d]); nullptr: f = 1.
constexpr int kSumCols = 32, kSumGroups = 32;
static __global__ void __launch_bounds__(kSumCols * kSumGroups)
column_sum_kernel(const float* part, float* out, long long rows, int D, const float* lam, float c) {
  __shared__ float s_sum[kSumGroups][kSumCols];
  const int j = threadIdx.x % kSumCols, q = threadIdx.x / kSumCols;
  const int col = blockIdx.x * kSumCols + j;
  float acc = 0.0f;
  if (col < D) {
    constexpr int U = 8;
    long long r = q;
    for (; r + (U - 1) * kSumGroups < rows; r += U * kSumGroups) {
      float v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) v[i] = part[(r + i * kSumGroups) * D + col];
#pragma unroll
      for (int i = 0; i < U; ++i) acc += v[i];
    }
    for (; r < rows; r += kSumGroups) acc += part[r * D + col];
  }
  s_sum[q][j] = acc;
  __syncthreads();
  if (q == 0 && col < D) {
    float t = 0.0f;
    for (int k = 0; k < kSumGroups; ++k) t += s_sum[k][j];
    out[col] = lam ? -c * sigm(lam[col]) * t : t;
  }
}

// One token for each of B requests: row b of u against the state in slot
// slots[b] (b itself without slots), updated in place. A slot outside
// [0, S) is a row without a request: zero output, no state touched. Bound by
// latency at the sizes that decoding has: one launch, C channels per lane.
template <class UT, int C>
__global__ void __launch_bounds__(256) gated_step_kernel(const UT* u, const float* lam, const int* slots,
                                                         float* state, UT* h, int B, int D, int S, float c) {
  const int nd = D / C;
  const long long k = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (k >= static_cast<long long>(B) * nd) return;
  const int b = static_cast<int>(k / nd), d = static_cast<int>(k - static_cast<long long>(b) * nd) * C;
  const int slot = slots ? slots[b] : b;
  const bool live = slot >= 0 && slot < S;
  URaw<UT, C> ur, ui, ux;
  const UT* ub = u + static_cast<long long>(b) * 3 * D + d;
  ur.load(ub);
  ui.load(ub + D);
  ux.load(ub + 2 * static_cast<long long>(D));
  float lv[C], sv[C], o[C];
  ld_f32<C>(lam + d, lv);
  float* sp = state + static_cast<long long>(live ? slot : 0) * D + d;
  ld_f32<C>(sp, sv);
#pragma unroll
  for (int q = 0; q < C; ++q) {
    const GateVal g = gate_values(ur.get(q), ui.get(q), decay_log2(lv[q], c));
    sv[q] = fmaf(g.a, sv[q], __builtin_amdgcn_sqrtf(g.v) * (g.i * ux.get(q)));
    o[q] = live ? sv[q] : 0.0f;
  }
  if (live) st_f32<C>(sp, sv);
  UT* hp = h + static_cast<long long>(b) * D + d;
  if constexpr (sizeof(UT) == 4) {
    st_f32<C>(reinterpret_cast<float*>(hp), o);
  } else if constexpr (C == 4) {
    *reinterpret_cast<u32x2*>(hp) = u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
  } else if constexpr (C == 2) {
    *reinterpret_cast<uint32_t*>(hp) = pack_bf16(o[0], o[1]);
  } else {
    hp->bits = static_cast<uint16_t>(pack_bf16(o[0], o[0]));
  }
}

}  // namespace pararnn
