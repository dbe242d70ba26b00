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
// chunks of 128 steps (4 / 128 bytes per element) are what the forward pass
// leaves for the adjoint, which rebuilds the others from u, in 32 bits: less
// to move than the states themselves, and not rounded to bf16.
#pragma once

#include "layer_common.h"

namespace pararnn {

constexpr int kGatedSave = 128;  // steps between two saved states

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
  unsigned long long* carry;  // [ngroups][slots] states at the groups' starts
  unsigned long long* agg;    // [nchunks][2][slots] chunk transforms
  unsigned int* ctr;        // [0] ticket
  int B, L, D, nchunks, ntiles_d, group;
  float c;
};

// Gate values of one step: v = 1 - a^2 = -expm1(2 log a) by its series where
// it is small (1 - a^2 itself would lose the digits that the subtraction
// cancels), m = sqrt(v) and 1/m from one reciprocal square root, 0 for both
// where v is 0. beta2: -c softplus(lam) log2(e).
struct GateVal {
  float r, i, a, m, im;
};
__device__ __forceinline__ GateVal gate_values(float ur, float ui, float beta2) {
  GateVal g;
  g.r = sigm(ur);
  g.i = sigm(ui);
  const float y = beta2 * g.r;  // log2 a
  g.a = __builtin_amdgcn_exp2f(y);
  const float w = y * -1.3862943611198906f;  // -2 log a >= 0
  float p = 1.0f / 5040.0f;  // (1 - exp(-w)) / w
  p = fmaf(p, w, -1.0f / 720.0f);
  p = fmaf(p, w, 1.0f / 120.0f);
  p = fmaf(p, w, -1.0f / 24.0f);
  p = fmaf(p, w, 1.0f / 6.0f);
  p = fmaf(p, w, -0.5f);
  p = fmaf(p, w, 1.0f);
  // from 0.25 on the cancellation costs under 2 bits; below it the series'
  // next term is under 2^-28
  const float v = w < 0.25f ? p * w : fmaf(-g.a, g.a, 1.0f);
  const float rs = __builtin_amdgcn_rsqf(v);
  g.im = v < 1.17549435e-38f ? 0.0f : rs;
  g.m = v * g.im;
  return g;
}

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

// The carry into a chunk. Chunks (counted in scan order) form groups of
// `group`. A chunk publishes its own transform as soon as it has it, except
// the last of a group, which publishes the state at its end: the next group's
// start. A chunk so waits for its group's start and for the transforms of the
// chunks before it in the group, and composes them in order: the chain of
// waits has one link per group, not per chunk, and the order of the sums does
// not depend on timing, so results repeat bit for bit. Tickets are taken
// chunk by chunk, so whatever a workgroup waits for has started before it.
// Words carry their tag (1: written) in the high half.
template <int C, bool RST>
__device__ __forceinline__ void chunk_carry(const GatedArgs& p, long long slots, long long chan, int cs, int q,
                                            const Lin<C, RST>& tot, float (&x)[C]) {
  const int grp = q / p.group, j = q - grp * p.group;
  const bool last = j == p.group - 1;
  if (!last && q < p.nchunks - 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      desc_put(p.agg + static_cast<long long>(q) * 2 * slots + chan + c * cs, 1u, tot.A[c]);
      desc_put(p.agg + (static_cast<long long>(q) * 2 + 1) * slots + chan + c * cs, 1u, tot.b[c]);
    }
  }
  Lin<C, RST> m;  // chunks before this one in the group, composed from the first on
  m.set_identity();
  for (int i = q - j; i < q; ++i) {
    unsigned long long wa[C], wb[C];
    while (true) {
      bool ok = true;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        wa[c] = desc_get(p.agg + static_cast<long long>(i) * 2 * slots + chan + c * cs);
        wb[c] = desc_get(p.agg + (static_cast<long long>(i) * 2 + 1) * slots + chan + c * cs);
        ok = ok && desc_ok(wa[c], 1u) && desc_ok(wb[c], 1u);
      }
      if (ok) break;
      __builtin_amdgcn_s_sleep(1);
    }
    Lin<C, RST> e;
#pragma unroll
    for (int c = 0; c < C; ++c) { e.A[c] = desc_val(wa[c]); e.b[c] = desc_val(wb[c]); }
    e.after(m);
    m = e;
  }
  if (grp > 0) {
    unsigned long long w[C];
    while (true) {
      bool ok = true;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        w[c] = desc_get(p.carry + static_cast<long long>(grp) * slots + chan + c * cs);
        ok = ok && desc_ok(w[c], 1u);
      }
      if (ok) break;
      __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = desc_val(w[c]);
  }
  m.apply(x);
  if (last && q < p.nchunks - 1) {
    float y[C];
#pragma unroll
    for (int c = 0; c < C; ++c) y[c] = x[c];
    tot.apply(y);
#pragma unroll
    for (int c = 0; c < C; ++c) desc_put(p.carry + static_cast<long long>(grp + 1) * slots + chan + c * cs, 1u, y[c]);
  }
}

// A workgroup of W waves covers LD * C channels (LD = 64 / LL lanes along D)
// and CL = W * LL * T steps: T steps in series per lane, a shuffle scan over
// the LL lane groups, an LDS scan over the waves, chunk_carry over the chunks.
template <class UT, int C, int T, int W, int LL, int OCC, bool RST>
__global__ void __launch_bounds__(64 * W, OCC) gated_scan_kernel(const GatedArgs p) {
  constexpr int LD = 64 / LL, CW = LD * C, CL = W * LL * T;
  __shared__ float s_A[W][CW], s_b[W][CW], s_carry[CW];
  __shared__ unsigned int s_ticket;

  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = tid >> 6;
  const int ld = lane % LD, ll = lane / LD;
  unsigned int ticket = blockIdx.x;
  if (p.nchunks > 1) {
    if (tid == 0) s_ticket = atomicAdd(p.ctr, 1u);
    __syncthreads();
    ticket = s_ticket;
  }
  const unsigned int ntiles = static_cast<unsigned int>(p.B) * p.ntiles_d;
  const int chunk = static_cast<int>(ticket / ntiles);
  const int tile = static_cast<int>(ticket - static_cast<unsigned int>(chunk) * ntiles);
  const int b = tile / p.ntiles_d;
  const int d0 = (tile - b * p.ntiles_d) * CW + ld * C;
  const bool dv = d0 < p.D;
  const int dc = dv ? d0 : 0;
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

  URaw<UT, C> uu[T][3];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int g = 0; g < 3; ++g) uu[t][g].load(ru, vu0 + t * ustep, static_cast<uint32_t>(g) * gstep);

  float beta2[C];
#pragma unroll
  for (int c = 0; c < C; ++c) beta2[c] = -1.4426950408889634f * p.c * softplus(p.lam[dc + c]);

  float A[T][C], x[T][C];  // x: input of the step, then nothing else
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const GateVal g = gate_values(uu[t][0].get(c), uu[t][1].get(c), beta2[c]);
      A[t][c] = g.a;
      x[t][c] = g.m * (g.i * uu[t][2].get(c));
    }
  if constexpr (RST) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const bool cut = l0 + t < p.L && p.reset[static_cast<long long>(b) * p.L + min(l0 + t, p.L - 1)] != 0;
#pragma unroll
      for (int c = 0; c < C; ++c) A[t][c] = cut ? __uint_as_float(kResetA) : A[t][c];
    }
  }
  const bool ragged = (chunk + 1) * static_cast<long long>(CL) > len;
  if (ragged) {  // steps past the length: identity
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
    for (int c = 0; c < C; ++c) { e.A[c] = A[t][c]; e.b[c] = x[t][c]; }
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
  if (wave == 0 && ll == 0) {
    float v[C];
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = (dv && p.h0) ? p.h0[static_cast<long long>(b) * p.D + dc + c] : 0.0f;
    if (dv && p.nchunks > 1) {
      Lin<C, RST> tot;
      tot.set_identity();
#pragma unroll
      for (int w = 0; w < W; ++w) {
        Lin<C, RST> e;
#pragma unroll
        for (int c = 0; c < C; ++c) { e.A[c] = s_A[w][ld * C + c]; e.b[c] = s_b[w][ld * C + c]; }
        e.after(tot);
        tot = e;
      }
      chunk_carry<C, RST>(p, static_cast<long long>(p.B) * p.ntiles_d * CW, static_cast<long long>(tile) * CW + ld,
                          LD, chunk, tot, v);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) s_carry[ld * C + c] = v[c];
  }
  __syncthreads();

  float h[C];
#pragma unroll
  for (int c = 0; c < C; ++c) h[c] = s_carry[ld * C + c];
  for (int w = 0; w < wave; ++w) {
    Lin<C, RST> e;
#pragma unroll
    for (int c = 0; c < C; ++c) { e.A[c] = s_A[w][ld * C + c]; e.b[c] = s_b[w][ld * C + c]; }
    e.apply(h);
  }
  if constexpr (LL > 1) excl.apply(h);
  if (p.saved && dv && l0 % kGatedSave == 0 && l0 < p.L)
    st_f32<C>(p.saved + (static_cast<long long>(l0 / kGatedSave) * p.B + b) * p.D + d0, h);

#pragma unroll
  for (int t = 0; t < T; ++t) {
    Lin<C, RST> e;
#pragma unroll
    for (int c = 0; c < C; ++c) { e.A[c] = A[t][c]; e.b[c] = x[t][c]; }
    e.apply(h);
    float o[C];
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = (ragged && l0 + t >= len) ? 0.0f : h[c];
    buf_st<UT, C>(rh, vh0 + t * gstep, 0u, o);  // dropped past L or D
  }
  if (p.hT && dv && chunk == p.nchunks - 1 && wave == W - 1 && ll == LL - 1)
    st_f32<C>(p.hT + static_cast<long long>(b) * p.D + d0, h);
}

// The adjoint of one chunk of CL = kGatedSave steps: a scan forward from the
// saved state for the h_{t-1}, and the scan backward for mu, on the same lanes.
template <class UT, int C, int T, int W, int LL, int OCC, bool RST>
__global__ void __launch_bounds__(64 * W, OCC) gated_adjoint_kernel(const GatedArgs p) {
  constexpr int LD = 64 / LL, CW = LD * C, CL = W * LL * T, NSEG = W * LL;
  static_assert(CL == kGatedSave, "a chunk starts at a saved state");
  __shared__ float s_A[W][CW], s_b[W][CW], s_B[W][CW], s_m[W][CW], s_carry[CW];
  __shared__ float s_dl[NSEG][CW];
  __shared__ unsigned int s_ticket;

  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = tid >> 6;
  const int ld = lane % LD, ll = lane / LD;
  unsigned int ticket = blockIdx.x;
  if (p.nchunks > 1) {
    if (tid == 0) s_ticket = atomicAdd(p.ctr, 1u);
    __syncthreads();
    ticket = s_ticket;
  }
  const unsigned int ntiles = static_cast<unsigned int>(p.B) * p.ntiles_d;
  const int rchunk = static_cast<int>(ticket / ntiles);
  const int chunk = p.nchunks - 1 - rchunk;  // taken from the end of L
  const int tile = static_cast<int>(ticket - static_cast<unsigned int>(rchunk) * ntiles);
  const int b = tile / p.ntiles_d;
  const int d0 = (tile - b * p.ntiles_d) * CW + ld * C;
  const bool dv = d0 < p.D;
  const int dc = dv ? d0 : 0;
  const int lt0 = (wave * LL + ll) * T;
  const int l0 = chunk * CL + lt0;
  const int len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
  const long long wrow = static_cast<long long>(b) * p.L + static_cast<long long>(chunk) * CL;
  const uint32_t gstep = static_cast<uint32_t>(p.D * sizeof(UT)), ustep = 3 * gstep;
  const uint32_t rows = static_cast<uint32_t>(min(p.L - chunk * CL, CL));
  constexpr uint32_t kOOB = 0x80000000u;
  const uint32_t vd = static_cast<uint32_t>(d0 * sizeof(UT));
  const uint32_t vu0 = dv ? static_cast<uint32_t>(lt0) * ustep + vd : kOOB;
  const uint32_t vh0 = dv ? static_cast<uint32_t>(lt0) * gstep + vd : kOOB;
  const __amdgpu_buffer_rsrc_t ru = make_rsrc(static_cast<const UT*>(p.u) + wrow * 3 * p.D, rows * ustep);
  const __amdgpu_buffer_rsrc_t rdh = make_rsrc(static_cast<const UT*>(p.dh) + wrow * p.D, rows * gstep);
  const __amdgpu_buffer_rsrc_t rdu = make_rsrc(static_cast<UT*>(p.du) + wrow * 3 * p.D, rows * ustep);

  URaw<UT, C> uu[T][3], gg[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
#pragma unroll
    for (int g = 0; g < 3; ++g) uu[t][g].load(ru, vu0 + t * ustep, static_cast<uint32_t>(g) * gstep);
    gg[t].load(rdh, vh0 + t * gstep, 0u);
  }
  float beta[C], beta2[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    beta[c] = -p.c * softplus(p.lam[dc + c]);
    beta2[c] = 1.4426950408889634f * beta[c];
  }

  float A[T][C], bb[T][C], dh[T][C];  // transform of the step; bb later holds h_{t-1}
  GateVal gv[T][C];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      gv[t][c] = gate_values(uu[t][0].get(c), uu[t][1].get(c), beta2[c]);
      A[t][c] = gv[t][c].a;
      bb[t][c] = gv[t][c].m * (gv[t][c].i * uu[t][2].get(c));
      dh[t][c] = gg[t].get(c);
    }
  if constexpr (RST) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const bool cut = l0 + t < p.L && p.reset[static_cast<long long>(b) * p.L + min(l0 + t, p.L - 1)] != 0;
#pragma unroll
      for (int c = 0; c < C; ++c) A[t][c] = cut ? __uint_as_float(kResetA) : A[t][c];
    }
  }
  const bool ragged = (chunk + 1) * static_cast<long long>(CL) > len;
  if (ragged) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        A[t][c] = l0 + t < len ? A[t][c] : 1.0f;
        bb[t][c] = l0 + t < len ? bb[t][c] : 0.0f;
        dh[t][c] = l0 + t < len ? dh[t][c] : 0.0f;
      }
  }

  // forward over the lane's steps, and backward: mu_t = A_t mu_{t+1} + A_t dh_t
  Lin<C, RST> fw, bw;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    Lin<C, RST> e;
#pragma unroll
    for (int c = 0; c < C; ++c) { e.A[c] = A[t][c]; e.b[c] = bb[t][c]; }
    if (t) e.after(fw);
    fw = e;
  }
#pragma unroll
  for (int t = T - 1; t >= 0; --t) {
    Lin<C, RST> e;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      e.A[c] = A[t][c];
      e.b[c] = (RST && __float_as_uint(A[t][c]) == kResetA) ? 0.0f : A[t][c] * dh[t][c];
    }
    if (t < T - 1) e.after(bw);
    bw = e;
  }
  Lin<C, RST> fx, bx;  // what precedes the lane in either direction, within the wave
  fx.set_identity();
  bx.set_identity();
  if constexpr (LL > 1) {
#pragma unroll
    for (int off = 1; off < LL; off *= 2) {
      const Lin<C, RST> prev = fw.shfl_up(off * LD);
      if (ll >= off) fw.after(prev);
      Lin<C, RST> next;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        next.A[c] = __shfl_down(bw.A[c], off * LD, 64);
        next.b[c] = __shfl_down(bw.b[c], off * LD, 64);
      }
      if (ll < LL - off) bw.after(next);
    }
    const Lin<C, RST> prev = fw.shfl_up(LD);
    if (ll > 0) fx = prev;
    Lin<C, RST> next;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      next.A[c] = __shfl_down(bw.A[c], LD, 64);
      next.b[c] = __shfl_down(bw.b[c], LD, 64);
    }
    if (ll < LL - 1) bx = next;
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
  if (wave == 0 && ll == 0) {
    float v[C];
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = (dv && p.dhT) ? p.dhT[static_cast<long long>(b) * p.D + dc + c] : 0.0f;
    if (dv && p.nchunks > 1) {
      Lin<C, RST> tot;
      tot.set_identity();
#pragma unroll
      for (int w = W - 1; w >= 0; --w) {
        Lin<C, RST> e;
#pragma unroll
        for (int c = 0; c < C; ++c) { e.A[c] = s_B[w][ld * C + c]; e.b[c] = s_m[w][ld * C + c]; }
        e.after(tot);
        tot = e;
      }
      chunk_carry<C, RST>(p, static_cast<long long>(p.B) * p.ntiles_d * CW, static_cast<long long>(tile) * CW + ld,
                          LD, rchunk, tot, v);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) s_carry[ld * C + c] = v[c];
  }
  // meanwhile the others rebuild their states from the saved one
  float h[C];
#pragma unroll
  for (int c = 0; c < C; ++c) h[c] = 0.0f;
  if (dv) ld_f32<C>(p.saved + (static_cast<long long>(chunk) * p.B + b) * p.D + d0, h);
  for (int w = 0; w < wave; ++w) {
    Lin<C, RST> e;
#pragma unroll
    for (int c = 0; c < C; ++c) { e.A[c] = s_A[w][ld * C + c]; e.b[c] = s_b[w][ld * C + c]; }
    e.apply(h);
  }
  if constexpr (LL > 1) fx.apply(h);
#pragma unroll
  for (int t = 0; t < T; ++t) {
    Lin<C, RST> e;
    float prev[C];
#pragma unroll
    for (int c = 0; c < C; ++c) { e.A[c] = A[t][c]; e.b[c] = bb[t][c]; prev[c] = h[c]; }
    e.apply(h);
#pragma unroll
    for (int c = 0; c < C; ++c) bb[t][c] = prev[c];
  }
  __syncthreads();
  float mu[C];
#pragma unroll
  for (int c = 0; c < C; ++c) mu[c] = s_carry[ld * C + c];
  for (int w = W - 1; w > wave; --w) {
    Lin<C, RST> e;
#pragma unroll
    for (int c = 0; c < C; ++c) { e.A[c] = s_B[w][ld * C + c]; e.b[c] = s_m[w][ld * C + c]; }
    e.apply(mu);
  }
  if constexpr (LL > 1) bx.apply(mu);

  float dl[C];
#pragma unroll
  for (int c = 0; c < C; ++c) dl[c] = 0.0f;
#pragma unroll
  for (int t = T - 1; t >= 0; --t) {
    const bool on = !ragged || l0 + t < len;
    float o[3][C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const GateVal v = gv[t][c];
      const float xv = uu[t][2].get(c), g = mu[c] + dh[t][c];
      const bool cut = RST && __float_as_uint(A[t][c]) == kResetA;
      const float prev = cut ? 0.0f : bb[t][c];
      const float ix = v.i * xv, gm = g * v.m;
      const float dla = g * v.a * fmaf(-ix * v.a, v.im, prev);
      dl[c] = on ? fmaf(dla, v.r, dl[c]) : dl[c];
      o[0][c] = on ? dla * beta[c] * fmaf(-v.r, v.r, v.r) : 0.0f;
      o[1][c] = on ? gm * (ix * (1.0f - v.i)) : 0.0f;
      o[2][c] = on ? gm * v.i : 0.0f;
      mu[c] = cut ? 0.0f : (on ? v.a * g : mu[c]);
    }
#pragma unroll
    for (int g = 0; g < 3; ++g)
      buf_st<UT, C, kBufNT>(rdu, vu0 + t * ustep, static_cast<uint32_t>(g) * gstep, o[g]);
  }
  if (p.dh0 && dv && l0 == 0) st_f32<C>(p.dh0 + static_cast<long long>(b) * p.D + d0, mu);
  if (p.dl_part) {  // summed over the lane groups in order
#pragma unroll
    for (int c = 0; c < C; ++c) s_dl[wave * LL + ll][ld * C + c] = dl[c];
    __syncthreads();
    if (wave == 0 && ll == 0 && dv) {
      float s[C];
#pragma unroll
      for (int c = 0; c < C; ++c) s[c] = 0.0f;
      for (int k = 0; k < NSEG; ++k)
#pragma unroll
        for (int c = 0; c < C; ++c) s[c] += s_dl[k][ld * C + c];
      st_f32<C>(p.dl_part + (static_cast<long long>(chunk) * p.B + b) * p.D + d0, s);
    }
  }
}

// out[d] = f(d) * sum of `rows` partial rows, in a fixed order: kSumGroups
// interleaved row groups per column, then the groups in turn.
// lam: f = -c s(lam[d]); nullptr: f = 1.
constexpr int kSumCols = 64, kSumGroups = 16;
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
    const GateVal g = gate_values(ur.get(q), ui.get(q), -1.4426950408889634f * c * softplus(lv[q]));
    sv[q] = fmaf(g.a, sv[q], g.m * (g.i * ux.get(q)));
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
