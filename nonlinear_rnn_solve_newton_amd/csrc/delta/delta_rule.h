// delta_rule.h -- gated delta rule over chunks of 64 steps, its adjoint, and
// its single-token step. Per value head, with S [dk][dv], unit q and k, decay a
// and write strength b (0 < b < 1):
//   S_t = a S_{t-1} + k b (v - a S_{t-1}^T k)^T,   o_t = scale S_t^T q.
//
// Within a chunk, with G_i the sum of log a over its first i steps, S0 the state
// in front of it and E_ij = exp(G_i - G_j) (zero where a document starts in
// between), the read values are X = V - diag(e^G) K S0 and
//   y = T X,  T = (1 + strictly lower(E_ij k_i.k_j b_j))^-1   (v less what k reads)
//   O = scale e^G Q S0 + P y,   P = lower(scale E_ij q_i.k_j b_j)
//   S1 = e^G_64 S0 + K^T (e^(G_64 - G) b y).
// T_ii = 1 and |T_ij| <= b_j <= 1 for i > j: a product of contractions between two unit keys. T
// is inverted by substitution in blocks of 16 and joined, never by its series,
// whose terms reach C(63, 31) for equal keys.
//
// delta_prep_kernel makes T, P and the rows' factors of all chunks at once;
// delta_scan_kernel carries the state, a wave per 16 columns of dv, which do not
// depend on each other. The adjoint carries dS back the same way,
//   dY = P^T dO + e^(G_64 - G) b K dS1,  dX = T^T dY = dV,
//   dS0 = e^G_64 dS1 + (scale e^G Q)^T dO - (e^G K)^T dX,
// and delta_grad_kernel takes the rest of all chunks at once:
//   dQ = scale e^G dO S0^T + D0 K,               D0_ij = scale E_ij b_j dO_i.y_j (i >= j)
//   dK read = D1 K - e^G dX S0^T,                D1_ij = -E_ij b_j dX_i.y_j      (i > j)
//   dK written = D0^T Q + D1^T K + e^(G_64 - G) b y dS1^T
//   b dL/db = k.(dK written),  which a gate's gradient (1 - b) b dL/db takes as it is.
// A step's log decay multiplies what passes it: with W_ij = D0_ij q_i.k_j + D1_ij k_i.k_j,
//   dL/dlog a_t = sum over j < t <= i of W_ij + sum over i >= t of what rows i read from S0
//               + sum over j < t of what rows j add to S1 + e^G_64 <S0, dS1>.
// (Row i's decayed terms less column i's, summed from the end, is the same in
// exact arithmetic, but a difference of large sums where decays are strong.)
#pragma once

#include "delta_common.h"

namespace pararnn {

constexpr int kDeltaChunk = 64;

struct DeltaView {  // [B][L][..], packed from the third dimension on; strides in elements
  const void* p;
  long long batch, token;
};

struct DeltaArgs {
  DeltaView q, k, v, gates;
  DeltaView gq, gk, gv, dgates;  // adjoint: outputs (gradients of q, k, v and the gates)
  const float* lam;              // [HV]
  const float* s0;               // [B][HV][dk][dv] or nullptr: the state in front; adjoint: dsT
  float* sT;                     // the state behind, or nullptr; adjoint: ds0
  void* o;                       // [B][L][HV][dv]; adjoint: dO
  const int* lengths;
  const uint8_t* reset;
  bf16x8* frags;                 // per chunk and value head: planes of T and P as operands
  float* rows;                   // per chunk and value head: kRows x 64 factors
  // As result tiles lie in registers, per chunk and value head [2 ceil(dv / 32)][tiles of 16 rows][64 lanes]:
  f32x4* states;                 // saved: the state in front of each chunk (2 ceil(dk / 32) tiles), or nullptr
  f32x4* ys;                     // saved: y (4 tiles)
  f32x4* dstates;                // adjoint: dS behind each chunk
  f32x4* dxs;                    // adjoint: dX
  float* dlam_part;              // adjoint: [HV][B chunks]
  // Of each segment, as the scans cross it: the state (adjoint: dS) that it puts out for none coming in, as result
  // tiles, and the matrix [DK][DK] that takes what comes in to what it adds to that
  f32x4* seg_add;
  float* seg_map;
  int B, L, H, HV, dk, dv, nc;
  int nseg, per;                 // segments, chunks of each
  float c, eps, scale;
  int wide, wide_qk;             // rows of bf16 o (adjoint: dV), and of dQ and dK, take 16-byte stores
};

// factors of a chunk's rows (NotR, NotB: 1 - s(gate) as s(-gate), which keeps its digits)
enum { kRowX = 0, kRowO = 1, kRowS = 2, kRowWhole = 3, kRowK = 4, kRowQ = 5, kRowB = 6, kRowG = 7, kRowR = 8,
       kRowSeg = 9, kRowNotR = 10, kRowNotB = 11, kRowGLow = 12, kRows = 13 };

// Blocks (16 rows x 32 inner indexes) of a lower triangular 64 x 64 operand,
// and of its transpose, that are not zero: 6 of 8
constexpr int kTriBlocks = 6;
__host__ __device__ constexpr int low_block(int i, int kb) { return i < 2 ? i : 2 + 2 * (i - 2) + kb; }
__host__ __device__ constexpr int up_block(int j, int kb) { return j < 2 ? 2 * j + kb : 4 + (j - 2); }
// operands per chunk, three planes of each: T's blocks, then P's
struct DeltaFrags {
  static constexpr int T = kTriBlocks * 3 * 64, ALL = 2 * T;
};

// tiles of 16 that n rows or columns take, in pairs
__host__ __device__ constexpr int delta_tiles(int n) { return (n + 31) / 32 * 2; }
// G_i - G_j of the sums of log a, in two floats each. Strong decays in front of weak ones leave sums of hundreds
// whose differences are of 0.1: from one float they, and the decays, are off by 2^-24 of the sums.
template <class V>
__device__ __forceinline__ V log_gap(V hi, V low, float hj, float lj) { return (hi - hj) + (low - lj); }
__device__ __forceinline__ int delta_len(const DeltaArgs& p, int b) {
  return p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
}
template <class UT>
__device__ __forceinline__ const UT* at(const DeltaView& v, int b, long long t) {
  return static_cast<const UT*>(v.p) + b * v.batch + t * v.token;
}
// n rows from step t on, from element d of the `packed` ones of a row
template <class UT>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const DeltaView& v, int b, long long t, int d, int n, int packed) {
  return make_rsrc(at<UT>(v, b, t) + d, static_cast<uint32_t>((n - 1) * v.token + packed - d) * sizeof(UT));
}
// where row `row` of a resource of rows `token` elements apart has its element d; nowhere unless `on`
template <class UT>
__device__ __forceinline__ uint32_t offset_of(int row, long long token, int d, bool on) {
  return on ? static_cast<uint32_t>((row * static_cast<int>(token) + d) * static_cast<int>(sizeof(UT))) : kNoLoad;
}
template <class UT>
__device__ __forceinline__ UT* out_at(const DeltaView& v, int b, long long t) {
  return static_cast<UT*>(const_cast<void*>(v.p)) + b * v.batch + t * v.token;
}

// 16 x 16 x 16 product in fp32: A from workgroup memory (row m, columns 4 g ..),
// B as a result tile holds it
__device__ __forceinline__ f32x4 mul16(const float* a, const f32x4& b, f32x4 c) {
  const f32x4 x = *reinterpret_cast<const f32x4*>(a);
#pragma unroll
  for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[s], b[s], c, 0, 0, 0);
  return c;
}

// Inverse of 1 + a for a strictly lower triangular block of 16 x 16 in workgroup
// memory: lane (m, g) solves column m of block g by substitution. The rows come
// in three parts, each read while the one before is worked on.
template <int ROW>
__device__ __forceinline__ void invert16(const float* a, int m, float (&x)[16]) {
  f32x4 r0[8], r1[13], r2[11];
  auto row = [&](int i, int j4) { return *reinterpret_cast<const f32x4*>(a + i * ROW + 4 * j4); };
#pragma unroll
  for (int i = 1; i <= 6; ++i) {
    if (i <= 4) r0[i - 1] = row(i, 0);
    else {
      r0[4 + 2 * (i - 5)] = row(i, 0);
      r0[5 + 2 * (i - 5)] = row(i, 1);
    }
  }
#pragma unroll
  for (int i = 7; i <= 11; ++i)
#pragma unroll
    for (int j = 0; j < (i + 3) / 4; ++j) r1[i <= 8 ? 2 * (i - 7) + j : 4 + 3 * (i - 9) + j] = row(i, j);
  x[0] = m == 0 ? 1.0f : 0.0f;
  auto solve = [&](int i, const f32x4* r) {
    float v = i == m ? 1.0f : 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < i) v = fmaf(-r[j >> 2][j & 3], x[j], v);
    x[i] = v;
  };
#pragma unroll
  for (int i = 1; i <= 6; ++i) solve(i, &r0[i <= 4 ? i - 1 : 4 + 2 * (i - 5)]);
#pragma unroll
  for (int i = 12; i <= 15; ++i)
#pragma unroll
    for (int j = 0; j < (i == 12 ? 3 : 4); ++j)
      if (i < 15) r2[i == 12 ? j : 3 + 4 * (i - 13) + j] = row(i, j);
#pragma unroll
  for (int i = 7; i <= 11; ++i) solve(i, &r1[i <= 8 ? 2 * (i - 7) : 4 + 3 * (i - 9)]);
#pragma unroll
  for (int j = 0; j < 4; ++j) r0[j] = row(15, j);
#pragma unroll
  for (int i = 12; i <= 14; ++i) solve(i, &r2[i == 12 ? 0 : 3 + 4 * (i - 13)]);
  solve(15, r0);
}

// A workgroup per chunk and value head: row factors, T and P (ADJ: their
// transposes) as operands of the scan, in memory order of its reads. A wave takes
// the 16 steps of tile w: of its queries, the products with the keys up to them,
// or (ADJ) of its keys, with the queries from them on. A lane then has 4 inner
// indexes of its row of P, as the operand wants them, and P never leaves
// registers; the keys' own products go to workgroup memory to be inverted, and at
// 36 KB four workgroups to a CU hide each other's substitution, the longest part.
// B = 8 L = 4096 H = 8, 128 wide, bf16: 74 us, 318 MB (4.3 TB/s; with P in workgroup
// memory it took 1.6 times as long); the adjoint's 91 us, 319 MB.
template <class UT, bool EVEN, int DK, bool ADJ>
__global__ void __launch_bounds__(256, sizeof(UT) == 2 ? 4 : 1) delta_prep_kernel(const DeltaArgs p) {
  constexpr int NP = DeltaPlanes<UT>::NP, KB = DK / 32, ROW = 68;
  __shared__ float sm[64 * ROW], st[64 * ROW];
  __shared__ float sg[64], sgl[64], sb[64], sseg[64], srk[64], srq[64];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), m = lane & 15, g = lane >> 4;
  const int ch = blockIdx.x % p.nc, bh = blockIdx.x / p.nc, b = bh / p.HV, hv = bh % p.HV, h = hv / (p.HV / p.H);
  const int t0 = ch * kDeltaChunk, len = delta_len(p, b);
  if (t0 >= len) return;
  const int n = min(len - t0, kDeltaChunk);
  float* rows = p.rows + (static_cast<long long>(bh) * p.nc + ch) * (kRows * 64);

  // own: the wave's 16 rows, column of the results; tile j of the others: their rows
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float nk = 0.0f, nq = 0.0f;
  {
    const int H = p.H * p.dk;
    const __amdgpu_buffer_rsrc_t kr = rows_of<UT>(p.k, b, t0, h * p.dk, n, H), qr = rows_of<UT>(p.q, b, t0, h * p.dk, n, H);
    const int i = 16 * w + m;
    // which tiles the wave multiplies with: the keys up to its own, or the queries (and keys) from it on
    auto other = [&](int j) { return ADJ ? j >= w : j <= w; };
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const int d = 32 * kb + 8 * g, count = p.dk - d;
      Piece<UT, EVEN> rk[4], rq[ADJ ? 4 : 1];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (other(j)) rk[j].load(kr, offset_of<UT>(16 * j + m, p.k.token, d, 16 * j + m < n && count > 0));
      if constexpr (ADJ) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (other(j)) rq[j].load(qr, offset_of<UT>(16 * j + m, p.q.token, d, 16 * j + m < n && count > 0));
      } else {
        rq[0].load(qr, offset_of<UT>(i, p.q.token, d, i < n && count > 0));
      }
      bf16x8 ok[NP], oq[NP], c[NP];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j == w) {
          planes_of(rk[j], count, ok);
          planes_of(rq[ADJ ? j : 0], count, oq);
        }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = plane_sum<NP>(ok, e), y = plane_sum<NP>(oq, e);
        nk = fmaf(x, x, nk);
        nq = fmaf(y, y, nq);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (other(j)) {
          planes_of(rk[j], count, c);
          mma<NP, NP>(kk[j], c, ok);
          if constexpr (ADJ) {
            planes_of(rq[j], count, c);
            mma<NP, NP>(qk[j], c, ok);
          } else {
            mma<NP, NP>(qk[j], c, oq);
          }
        }
    }
  }
  nk += __shfl_xor(nk, 16, 64);
  nk += __shfl_xor(nk, 32, 64);
  nq += __shfl_xor(nq, 16, 64);
  nq += __shfl_xor(nq, 32, 64);
  if (g == 0) {
    srk[16 * w + m] = 1.0f / sqrtf(nk + p.eps);
    srq[16 * w + m] = 1.0f / sqrtf(nq + p.eps);
  }
  if (w == (ADJ ? 3 : 0)) {  // the gates: a lane per step, in the wave with the fewest products
    const int i = lane;
    const bool on = i < n;
    const UT* gp = at<UT>(p.gates, b, t0 + min(i, n - 1)) + hv;
    const float ga = load1(gp), gb = load1(gp + p.HV);
    const float r = on ? sigm(ga) : 0.0f, beta = on ? sigm(gb) : 0.0f;
    const float coef = -p.c * softplus(p.lam[hv]);
    // e^-1024 is 0 beside any float: held there, no sum is infinite
    const float la = coef * r;
    double sum = on ? (la < -1024.0f ? -1024.0f : la) : 0.0f;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double u = __shfl_up(sum, o, 64);
      if (i >= o) sum += u;
    }
    const float G = static_cast<float>(sum), low = static_cast<float>(sum - static_cast<double>(G));
    const bool start = on && p.reset && p.reset[static_cast<long long>(b) * p.L + t0 + i] != 0;
    const unsigned long long starts = __ballot(start);
    const int seg = __popcll(starts & (~0ull >> (63 - i)));
    sg[i] = G;
    sgl[i] = low;
    sb[i] = beta;
    sseg[i] = static_cast<float>(seg);
    rows[kRowB * 64 + i] = beta;
    rows[kRowG * 64 + i] = G;
    rows[kRowGLow * 64 + i] = low;
    rows[kRowR * 64 + i] = r;
    rows[kRowSeg * 64 + i] = static_cast<float>(seg);
    rows[kRowNotR * 64 + i] = on ? sigm(-ga) : 0.0f;
    rows[kRowNotB * 64 + i] = on ? sigm(-gb) : 0.0f;
  }
  __syncthreads();
  constexpr float kLog2e = 1.4426950408889634f;
  bf16x8* const out = p.frags + (static_cast<long long>(bh) * p.nc + ch) * DeltaFrags::ALL;
  // The first step whose key or gates are no numbers (a key's length is a positive one else). Rows from there on
  // stay out of T and P, whose zeros above the diagonal would carry them to the rows in front; the scan has them
  // from kRowX. (The adjoint's gradients run the other way as well, and are not kept apart.)
  int good = 64;
  if constexpr (!ADJ) {
    const unsigned long long bad = __ballot(!(srk[lane] > 0.0f) || sg[lane] != sg[lane] || sb[lane] != sb[lane]);
    good = bad ? __builtin_ctzll(bad) : 64;
  }
  {
    // element (row i, column j) of both: E_ij with the lengths, b_j and the scale. The lane's own index is the
    // row i (ADJ: the column j), and it has 4 of the other.
    const int own = 16 * w + m;
    const float Go = sg[own], lo = sgl[own], so = sseg[own], ko = srk[own], qo = srq[own] * p.scale, bo = sb[own];
    const bool live = own < good;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x4 mv = {0.0f, 0.0f, 0.0f, 0.0f};
      if (ADJ ? j >= w : j <= w) {
        const int c = 16 * j + 4 * g;
        const f32x4 Gc = *reinterpret_cast<const f32x4*>(&sg[c]), sc = *reinterpret_cast<const f32x4*>(&sseg[c]);
        const f32x4 gap = log_gap(Gc, *reinterpret_cast<const f32x4*>(&sgl[c]), Go, lo);  // columns' less the own
        const f32x4 kc = *reinterpret_cast<const f32x4*>(&srk[c]);
        const f32x4 fc = *reinterpret_cast<const f32x4*>(ADJ ? &srq[c] : &sb[c]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = ADJ ? c + e : own, col = ADJ ? own : c + e;
          const bool low = row >= col && sc[e] == so && live;
          const float x = low ? __builtin_amdgcn_exp2f((ADJ ? gap[e] : -gap[e]) * kLog2e) : 0.0f;
          // k_i k_j b_j and scale q_i k_j b_j
          const float y = x * kc[e] * ko * (ADJ ? bo : fc[e]);
          mv[e] = row > col && live ? y * kk[j][e] : 0.0f;
          qk[j][e] = ADJ || low ? qk[j][e] * (ADJ ? x * p.scale * fc[e] * ko * bo : x * kc[e] * fc[e] * qo) : 0.0f;
        }
      } else {
        qk[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
      if constexpr (ADJ) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sm[(16 * j + 4 * g + e) * ROW + own] = mv[e];
      } else {
        *reinterpret_cast<f32x4*>(&sm[own * ROW + 16 * j + 4 * g]) = mv;
      }
      if (ADJ ? j < w : j > w) {  // above the diagonal
#pragma unroll
        for (int e = 0; e < 4; ++e) st[(ADJ ? 16 * j + 4 * g + e : own) * ROW + (ADJ ? own : 16 * j + 4 * g + e)] = 0.0f;
      }
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
      if (ADJ ? kb >= w / 2 : kb <= w / 2) {
        bf16x8 o[3];
        split_tiles<3>(qk[2 * kb], qk[2 * kb + 1], o);
        const int id = ADJ ? up_block(w, kb) : low_block(w, kb);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) out[DeltaFrags::T + (id * 3 + pl) * 64 + lane] = o[pl];
      }
  }
  __syncthreads();
  if (w == 0) {  // the four diagonal blocks
    float x[16];
    invert16<ROW>(sm + 16 * g * ROW + 16 * g, m, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) st[(16 * g + i) * ROW + 16 * g + m] = x[i];
  } else if (w == 1) {
    const int i = lane;
    const float G = sg[i], Ge = sg[63], se = sseg[63], rest = log_gap(Ge, sgl[63], G, sgl[i]);
    const float gamma = sseg[i] == 0.0f ? __builtin_amdgcn_exp2f(G * kLog2e) : 0.0f;
    const float tail = sseg[i] == se ? __builtin_amdgcn_exp2f(rest * kLog2e) : 0.0f;
    rows[kRowX * 64 + i] = i < good ? gamma * srk[i] : __uint_as_float(0x7fc00000u);
    rows[kRowO * 64 + i] = p.scale * gamma * srq[i];
    rows[kRowS * 64 + i] = tail * srk[i] * sb[i];
    rows[kRowWhole * 64 + i] = se == 0.0f ? __builtin_amdgcn_exp2f(Ge * kLog2e) : 0.0f;
    rows[kRowK * 64 + i] = srk[i];
    rows[kRowQ * 64 + i] = srq[i];
  }
  __syncthreads();
#pragma unroll
  for (int d = 1; d < 4; ++d) {  // the blocks below: T_ij = -T_ii (sum of M_ik T_kj over j <= k < i)
    if (w >= d) {
      const int j = w - d;
      f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < d; ++k) {
        f32x4 t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = st[(16 * (j + k) + 4 * g + e) * ROW + 16 * j + m];
        s = mul16(sm + (16 * w + m) * ROW + 16 * (j + k) + 4 * g, t, s);
      }
      const f32x4 r = mul16(st + (16 * w + m) * ROW + 16 * w + 4 * g, s, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
      for (int e = 0; e < 4; ++e) st[(16 * w + 4 * g + e) * ROW + 16 * j + m] = -r[e];
    }
    __syncthreads();
  }
  for (int id = w; id < kTriBlocks; id += 4) {
    const int i = ADJ ? (id < 4 ? id / 2 : id - 2) : id < 2 ? id : 2 + (id - 2) / 2;
    const int kb = ADJ ? (id < 4 ? id % 2 : 1) : id < 2 ? 0 : (id - 2) % 2;
    float x[8];
#pragma unroll
    for (int h2 = 0; h2 < 2; ++h2) {
      const int c = 32 * kb + 16 * h2 + 4 * g, r = 16 * i + m;
      if constexpr (ADJ) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * h2 + e] = st[(c + e) * ROW + r];
      } else {
        const f32x4 v = *reinterpret_cast<const f32x4*>(&st[r * ROW + c]);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * h2 + e] = v[e];
      }
    }
    bf16x8 o[3];
    split8<3>(x, o);
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) out[(id * 3 + pl) * 64 + lane] = o[pl];
  }
}

// What a chunk brings into workgroup memory for the scans; VC: columns of v
// (dO) that the workgroup takes. Where the tensors are bf16, a wave leaves its
// results in the place of its own columns of v, and they go out by whole rows
// while the next chunk is worked on. KONLY: neither q nor P.
template <class UT, int DK, int VC, bool ADJ, bool KONLY>
struct DeltaBuf {
  static constexpr int NP = DeltaPlanes<UT>::NP;
  static constexpr int FA = KONLY ? DeltaFrags::T : DeltaFrags::ALL;  // of the chunk's triangular operands
  DeltaTile<DK, NP> k;
  DeltaTile<KONLY ? 32 : DK, NP, KONLY ? 1 : 64> q;
  DeltaTile<VC, NP> v;
  bf16x8 frags[FA];
  float rows[4 * 64];
};

// The scans' common part. NW waves have 16 NC columns of dv each and work on a
// chunk; NL more waves bring the next one meanwhile and send the results of the
// one before. A CU takes 25 bytes a cycle from memory, so that a chunk (77 KB)
// keeps whoever asks for it waiting for 3000 cycles of the 5500 that its products
// take (with each wave loading its share, 8500). One such wave does where loads
// write to workgroup memory (kDirect), four where they pass through registers;
// fp32 needs the registers of two waves for one, and its waves load for
// themselves. Eight waves that each load a share of a chunk of 128 columns, two on
// a SIMD, take 10 us for it, two workgroups of four 7.5.
//
// B = 8 L = 4096 H = 8, 128 wide, bf16, with what the adjoint needs: 281 us forward,
// 297 back (910 and 886 MB, half of them the fp32 states and y, or dS and dX, going out;
// 3.0 to 3.2 TB/s); a chunk of a workgroup takes 4.4 us, 3.4 where no states go out,
// of which the matrix instructions are 1.2. The chain of a chunk's products bounds it.
//
// Few heads leave CUs idle, so a sequence is cut into segments. What a segment
// makes of the state in front of it is affine: delta_segment_kernel (SEG) scans
// all segments at once for the state that each adds, and with the columns of the
// identity and no v for the matrix; the scans then start every segment from the
// product over those before it. B = 1 L = 65536 H = 16: 480 to 560 us for the segments, 530 to
// 630 for the scan (1.9 GB, 3.0 to 3.6 TB/s), which took 2650 in one piece.
template <class UT, int MODE, int DK, int NC, int NW, bool ADJ, bool SEG = false>
struct DeltaScan {
  static constexpr int NP = DeltaPlanes<UT>::NP, RT = DK / 16, KB = DK / 32, VC = 16 * NC * NW;
  static constexpr bool DIRECT = MODE == kDirect, INPLACE = sizeof(UT) == 2;
  static constexpr int NL = DIRECT ? 1 : INPLACE ? 4 : 0, THREADS = 64 * (NW + NL), NT = 64 * (NL ? NL : NW);
  static constexpr bool SEGMENT = SEG, KONLY = SEG && !ADJ;
  typedef DeltaBuf<UT, DK, VC, ADJ, KONLY> Buf;
  static constexpr int NBUF = 2 * sizeof(Buf) <= 160 * 1024 ? 2 : 1;
  static_assert(NL == 0 || NBUF == 2, "a buffer to work on and one to fill");
  // rounds of the loading threads: chunks of q or k, of v, of the triangular operands, row factors
  static constexpr int TP = 64 * DK / 8 / NT, CP = 64 * VC / 8 / NT, FP = (Buf::FA + NT - 1) / NT, VP = 256 / NT;
  static_assert(64 * DK / 8 % NT == 0 && 256 % NT == 0 && 64 * VC / 8 % NT == 0 && DeltaFrags::ALL % 64 == 0, "whole rounds");

  // A tensor's rows of the chunk that is fetched next. Rows behind a row's last step lie past the resource's
  // extent (a token is at least as long as its packed elements) and so come as zeros: nothing but the
  // resource changes from chunk to chunk.
  struct Source {
    const char* at;      // the chunk's first row
    long long step;      // bytes from chunk to chunk
    uint32_t row, tail;  // bytes from row to row, and of a row's elements that may be read
    __device__ __forceinline__ void set(const DeltaView& v, int b, long long t, int d, int packed, int dir) {
      row = static_cast<uint32_t>(v.token) * sizeof(UT);
      at = reinterpret_cast<const char*>(pararnn::at<UT>(v, b, t) + d);
      step = dir * static_cast<long long>(row) * kDeltaChunk;
      tail = static_cast<uint32_t>(packed - d) * sizeof(UT);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(int n) const { return make_rsrc(at, (n - 1) * row + tail); }
  };

  const DeltaArgs& p;
  int lane, w, m, g, b, hv, h, bh, wg0, col0, cols, len, seg, c0, nch;  // chunks c0 to c0 + nch - 1
  bool idle, loads, last, ident;  // last: no chunks behind the segment's; ident: columns of the identity
  // of the loading threads
  int lt, dir, left;  // number, direction, steps of the chunk that is fetched next
  Source sk, sq, sv;
  const bf16x8* fp;
  const float* rp;
  Piece<UT, MODE != kOdd> rk[DIRECT ? 1 : TP], rq[DIRECT ? 1 : TP], rv[DIRECT ? 1 : CP];
  i32x4 rf[DIRECT ? 1 : FP];
  float rr[VP];

  // v: the tensor whose columns the waves have; dir: 1 from the first chunk on, -1 from the last
  __device__ __forceinline__ DeltaScan(const DeltaArgs& a, const DeltaView& v, int dir_) : p(a), dir(dir_) {
    const int tid = threadIdx.x;
    lane = tid & 63;
    w = __builtin_amdgcn_readfirstlane(tid >> 6);
    m = lane & 15;
    g = lane >> 4;
    // the slices of a segment follow each other on one XCD, whose L2 holds its chunk
    const int nslv = (p.dv + VC - 1) / VC, nsl = SEG ? nslv + (p.dk + VC - 1) / VC : nslv;
    const int x = blockIdx.x % 8, l = blockIdx.x / 8, unit = (l / nsl) * 8 + x;
    idle = unit >= p.B * p.HV * p.nseg;
    bh = unit % (p.B * p.HV);
    seg = idle ? 0 : unit / (p.B * p.HV);
    b = bh / p.HV;
    hv = bh % p.HV;
    h = hv / (p.HV / p.H);
    ident = SEG && l % nsl >= nslv;
    wg0 = (l % nsl - (ident ? nslv : 0)) * VC;
    col0 = wg0 / 16 + w * NC;
    cols = ident ? p.dk : p.dv;
    len = delta_len(p, b);
    const int all = (len + kDeltaChunk - 1) / kDeltaChunk;
    c0 = seg * p.per;
    nch = max(min(all - c0, p.per), 0);
    last = c0 + nch >= all;
    idle = idle || (seg > 0 && nch == 0);  // the first segment takes rows without steps
    if (SEG) {  // what nothing comes after or before in the scan's order
      const bool end = ADJ ? seg == 0 : last, start = ADJ ? last : seg == 0;
      idle = idle || end || (ident && start);
    }
    loads = NL && w >= NW;
    lt = NL ? tid - 64 * NW : tid;
    const int first = dir > 0 || nch == 0 ? c0 : c0 + nch - 1;
    left = len - first * kDeltaChunk;
    sk.set(p.k, b, static_cast<long long>(first) * kDeltaChunk, h * p.dk, p.H * p.dk, dir);
    sq.set(p.q, b, static_cast<long long>(first) * kDeltaChunk, h * p.dk, p.H * p.dk, dir);
    sv.set(v, b, static_cast<long long>(first) * kDeltaChunk, hv * p.dv, p.HV * p.dv, dir);
    fp = p.frags + (static_cast<long long>(bh) * p.nc + first) * DeltaFrags::ALL;
    rp = p.rows + (static_cast<long long>(bh) * p.nc + first) * (kRows * 64);
  }
  // the lane's column of v: column m of tile col0 + cc
  __device__ __forceinline__ int col(int cc) const { return delta_label(col0 + cc, m); }
  // a tile of COLS columns, those from d0 on of `cols`
  template <int COLS, int N, class Regs>
  __device__ __forceinline__ void fetch_tile(const Source& x, int d0, int cols, DeltaTile<COLS, NP>& to, Regs& r) {
    constexpr int CH = COLS / 8;
    const __amdgpu_buffer_rsrc_t rs = x.rows(min(left, kDeltaChunk));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lt + NT * i, d = d0 + DeltaTile<COLS, NP>::source(e);
      const uint32_t off = d < cols ? static_cast<uint32_t>(e / CH) * x.row + d * static_cast<uint32_t>(sizeof(UT)) : kNoLoad;
      if constexpr (DIRECT) load_to_lds(rs, &to.x[0][(NT * i + (lt & ~63)) * 8], off);
      else r[i].load(rs, off);
    }
  }
  // the next chunk's loads
  __device__ __forceinline__ void fetch(Buf& to) {
    fetch_tile<DK, TP>(sk, 0, p.dk, to.k, rk);
    if constexpr (!KONLY) fetch_tile<DK, TP>(sq, 0, p.dk, to.q, rq);
    fetch_tile<VC, CP>(sv, wg0, ident ? 0 : p.dv, to.v, rv);
    const __amdgpu_buffer_rsrc_t fr = make_rsrc(fp, Buf::FA * 16);
#pragma unroll
    for (int i = 0; i < FP; ++i) {
      if constexpr (DIRECT) {
        if (NT * (i + 1) <= Buf::FA || (lt & ~63) + NT * i < Buf::FA) load_to_lds(fr, &to.frags[(lt & ~63) + NT * i], (lt + NT * i) * 16);
      } else {
        rf[i] = __builtin_amdgcn_raw_buffer_load_b128(fr, (lt + NT * i) * 16, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < VP; ++i) rr[i] = rp[lt + NT * i];
    sk.at += sk.step;
    sq.at += sq.step;
    sv.at += sv.step;
    fp += dir * DeltaFrags::ALL;
    rp += dir * (kRows * 64);
    left -= dir * kDeltaChunk;
  }
  // what came through registers; then the loads that did not are waited for
  __device__ __forceinline__ void land(Buf& to) {
    if constexpr (!DIRECT) {
      bf16x8 o[NP];
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        planes_of(rk[i], p.dk - DeltaTile<DK, NP>::source(lt + NT * i), o);
        to.k.put_slot(lt + NT * i, o);
      }
#pragma unroll
      for (int i = 0; i < (KONLY ? 0 : TP); ++i) {
        planes_of(rq[i], p.dk - DeltaTile<DK, NP>::source(lt + NT * i), o);
        to.q.put_slot(lt + NT * i, o);
      }
#pragma unroll
      for (int i = 0; i < CP; ++i) {
        planes_of(rv[i], (ident ? 0 : p.dv) - wg0 - DeltaTile<VC, NP>::source(lt + NT * i), o);
        to.v.put_slot(lt + NT * i, o);
      }
#pragma unroll
      for (int i = 0; i < FP; ++i)
        if (NT * (i + 1) <= Buf::FA || lt + NT * i < Buf::FA) to.frags[lt + NT * i] = __builtin_bit_cast(bf16x8, rf[i]);
    }
#pragma unroll
    for (int i = 0; i < VP; ++i) to.rows[lt + NT * i] = rr[i];
    if constexpr (DIRECT) __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  }
  // rows of a chunk in memory, and of those the ones with steps: zeros behind them, whatever the others are
  __device__ __forceinline__ int rows_of_chunk(int ch) const { return min(p.L - ch * kDeltaChunk, kDeltaChunk); }
  __device__ __forceinline__ int live_of_chunk(int ch) const { return len - ch * kDeltaChunk; }
  // The wave's results Y of a chunk, rows of [..][HV][dv]: into the place of its columns of v, to be sent later, or
  // straight to memory
  __device__ __forceinline__ void result(Buf& u, const DeltaView& to, int ch, const f32x4 (&Y)[NC][4]) const {
    if constexpr (INPLACE) {
#pragma unroll
      for (int cc = 0; cc < NC; ++cc)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            u.v.x[0][u.v.pos(16 * i + 4 * g + r, delta_label(w * NC + cc, m))] = static_cast<__bf16>(Y[cc][i][r]);
    } else {
      const int rows = rows_of_chunk(ch), live = live_of_chunk(ch);
      UT* o = out_at<UT>(to, b, static_cast<long long>(ch) * kDeltaChunk) + static_cast<long long>(hv) * p.dv;
#pragma unroll
      for (int cc = 0; cc < NC; ++cc)
        if (col(cc) < p.dv) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (16 * i + 4 * g + r < rows)
                store1(o + (16 * i + 4 * g + r) * to.token + col(cc), 16 * i + 4 * g + r < live ? Y[cc][i][r] : 0.0f);
        }
    }
  }
  // The results of a chunk out of its buffer, by the loading waves: each takes the slots that it fills next, so
  // nobody overwrites what another wave has not taken yet.
  __device__ __forceinline__ void send(const Buf& u, const DeltaView& to, int ch) const {
    if constexpr (INPLACE) {
      const int rows = rows_of_chunk(ch), live = live_of_chunk(ch);
      i32x4 v[CP];
#pragma unroll
      for (int i = 0; i < CP; ++i) v[i] = *reinterpret_cast<const i32x4*>(&u.v.x[0][(lt + NT * i) * 8]);
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): taken, before a load may write there
      bf16* o = reinterpret_cast<bf16*>(out_at<UT>(to, b, static_cast<long long>(ch) * kDeltaChunk)) +
                static_cast<long long>(hv) * p.dv + wg0;
#pragma unroll
      for (int i = 0; i < CP; ++i) {
        const int e = lt + NT * i, row = e / (VC / 8), d = DeltaTile<VC, NP>::source(e), count = p.dv - wg0 - d;
        bf16* at = o + row * to.token + d;
        if (row >= live) v[i] = i32x4{0, 0, 0, 0};
        if (row < rows && count > 0) {
          if (p.wide) {  // dv is a multiple of 8
            *reinterpret_cast<i32x4*>(at) = v[i];
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < count) at[k].bits = static_cast<uint16_t>(static_cast<uint32_t>(v[i][k >> 1]) >> (16 * (k & 1)));
          }
        }
      }
    }
  }
  __device__ __forceinline__ f32x4 row4(const Buf& u, int kind, int i) const {
    return *reinterpret_cast<const f32x4*>(&u.rows[kind * 64 + 16 * i + 4 * g]);
  }
  // [dk][dv] fp32 matrices as the wave's tiles
  __device__ __forceinline__ void load_state(const float* s, f32x4 (&S)[NC][RT]) const {
#pragma unroll
    for (int cc = 0; cc < NC; ++cc)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = delta_label(t, 4 * g + r);
          S[cc][t][r] = s && row < p.dk && col(cc) < p.dv ? s[static_cast<long long>(row) * p.dv + col(cc)] : 0.0f;
        }
  }
  __device__ __forceinline__ void store_state(float* s, const f32x4 (&S)[NC][RT]) const {
#pragma unroll
    for (int cc = 0; cc < NC; ++cc)
      if (col(cc) < p.dv) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = delta_label(t, 4 * g + r);
            if (row < p.dk) s[static_cast<long long>(row) * p.dv + col(cc)] = S[cc][t][r];
          }
      }
  }
  // What the segments in front of this one in the scan's order (ADJ: behind it) make of `start`
  __device__ __forceinline__ void join(const float* start, f32x4 (&S)[NC][RT]) const {
    const int nct = delta_tiles(p.dv), all = (len + kDeltaChunk - 1) / kDeltaChunk;
    const int from = ADJ ? (all + p.per - 1) / p.per - 1 : 0;  // the one that starts from `start` itself
    if (all == 0 || seg == from) {
      load_state(start, S);
      return;
    }
    for (int e = from; e != seg; e += ADJ ? -1 : 1) {
      const long long unit = static_cast<long long>(bh) * p.nseg + e;
      const float* map = p.seg_map + unit * (DK * DK);
      f32x4 N[NC][RT];
#pragma unroll
      for (int cc = 0; cc < NC; ++cc)
#pragma unroll
        for (int t = 0; t < RT; ++t)
          N[cc][t] = col0 + cc < nct ? p.seg_add[((unit * nct + col0 + cc) * RT + t) * 64 + lane] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (e != from) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          bf16x8 sb[NC][3];
#pragma unroll
          for (int cc = 0; cc < NC; ++cc) split_tiles<3>(S[cc][2 * kb], S[cc][2 * kb + 1], sb[cc]);
#pragma unroll
          for (int t0 = 0; t0 < RT; t0 += 4) {
            bf16x8 a[4][3];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const f32x4* r = reinterpret_cast<const f32x4*>(map + delta_label(t0 + t, m) * DK + 32 * kb + 8 * g);
              split_tiles<3>(r[0], r[1], a[t]);
            }
#pragma unroll
            for (int cc = 0; cc < NC; ++cc) {
              f32x4(&c)[4] = *reinterpret_cast<f32x4(*)[4]>(&N[cc][t0]);
              mma_rows<3, 3>(c, a, sb[cc]);
            }
          }
        }
      }
#pragma unroll
      for (int cc = 0; cc < NC; ++cc)
#pragma unroll
        for (int t = 0; t < RT; ++t) S[cc][t] = N[cc][t];
    }
  }
  // SEG: the identity's columns, and what became of them or of the state's
  __device__ __forceinline__ void identity(f32x4 (&S)[NC][RT]) const {
#pragma unroll
    for (int cc = 0; cc < NC; ++cc)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = delta_label(t, 4 * g + r);
          S[cc][t][r] = row == col(cc) && row < p.dk ? 1.0f : 0.0f;
        }
  }
  __device__ __forceinline__ void store_segment(const f32x4 (&S)[NC][RT]) const {
    const long long unit = static_cast<long long>(bh) * p.nseg + seg;
    if (!ident) {
      store_tiles<0, RT>(p.seg_add, unit, RT, S);
      return;
    }
#pragma unroll
    for (int cc = 0; cc < NC; ++cc)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) p.seg_map[unit * (DK * DK) + delta_label(t, 4 * g + r) * DK + col(cc)] = S[cc][t][r];
  }
  // tiles [FROM, TO) of each of the wave's columns as they lie, n of them per column tile in memory
  template <int FROM, int TO, int N>
  __device__ __forceinline__ void store_tiles(f32x4* to, long long id, int n, const f32x4 (&Y)[NC][N]) const {
    const int nct = delta_tiles(p.dv), c0 = col0;
#pragma unroll
    for (int cc = 0; cc < NC; ++cc)
      if (c0 + cc < nct) {
        f32x4* at = to + ((id * nct + c0 + cc) * n) * 64 + lane;
#pragma unroll
        for (int t = FROM; t < TO; ++t)
          if (t < n) at[t * 64] = Y[cc][t];
      }
  }
};

// y += a x for a triangular a given by its blocks: lower, or (UP) the transpose
// of one. XP: planes that x has room for, NB: those that count.
template <int NA, int NB, int NC, bool UP = false, int XP>
__device__ __forceinline__ void tri_rows(f32x4 (&y)[NC][4], const bf16x8 (&a)[kTriBlocks][NA], const bf16x8 (&x)[NC][2][XP]) {
  constexpr int N = NA > NB ? NA : NB;
#pragma unroll
  for (int s = N - 1; s >= 0; --s)
#pragma unroll
    for (int k = 0; k <= s; ++k)
      if (k < NA && s - k < NB) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (UP ? kb >= i / 2 : kb <= i / 2) {
#pragma unroll
              for (int cc = 0; cc < NC; ++cc)
                y[cc][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[UP ? up_block(i, kb) : low_block(i, kb)][k], x[cc][kb][s - k],
                                                                   y[cc][i], 0, 0, 0);
            }
      }
}

// TG tiles of the state from t0 on: S += a x over the chunk's rows
template <int NP, int TG, int NC, int RT>
__device__ __forceinline__ void state_tiles(f32x4 (&S)[NC][RT], int t0, const bf16x8 (&a)[TG][2][NP], const bf16x8 (&x)[NC][2][3]) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int k = 0; k <= s; ++k)
      if (k < NP) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int t = 0; t < TG; ++t)
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
              S[cc][t0 + t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][kb][k], x[cc][kb][s - k], S[cc][t0 + t], 0, 0, 0);
      }
}

// Rows of a wave's chunk from the first one on whose value is no number. They are kept from T's and P's products,
// whose zeros above the diagonal would carry them to the rows in front (0 times a NaN is one), and then are NaN.
struct DeltaBadRows {
  int first;  // of the lane's column
  static __device__ __forceinline__ int row(int i, int g, int r) { return 16 * i + 4 * g + r; }
  // from the operand of the values read, whose rows from `first` on become zeros; the lanes of a column agree
  __device__ __forceinline__ void take(bf16x8 (&x)[2][3], int g) {
    first = 64;
    i32x4 w[2][3];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) w[kb][pl] = __builtin_bit_cast(i32x4, x[kb][pl]);
#pragma unroll
    for (int e = 15; e >= 0; --e) {  // element e: row e % 4 of the lane's in tile e / 4
      const int u = w[e >> 3][0][(e & 7) >> 1], bits = e & 1 ? u >> 16 : u;
      if ((bits & 0x7f80) == 0x7f80) first = row(e >> 2, g, e & 3);
    }
    first = min(first, __shfl_xor(first, 16, 64));
    first = min(first, __shfl_xor(first, 32, 64));
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 8 * kb + 2 * i, r = row(e >> 2, g, e & 3);
        const int keep = r + 1 < first ? -1 : r < first ? 0xffff : 0;
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) w[kb][pl][i] &= keep;
      }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) x[kb][pl] = __builtin_bit_cast(bf16x8, w[kb][pl]);
  }
  __device__ __forceinline__ void mark(f32x4 (&y)[4], int g) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) y[i][r] = row(i, g, r) >= first ? __uint_as_float(0x7fc00000u) : y[i][r];
  }
};

// A chunk of the scan
template <class D, class UT, int DK, int NC>
__device__ __forceinline__ void delta_scan_chunk(const D& s, const DeltaArgs& p, const DeltaView& o, int ch, typename D::Buf& u,
                                                 f32x4 (&S)[NC][D::RT], bf16x8 (&sb)[NC][D::KB][3]) {
  constexpr int NP = D::NP, RT = D::RT, KB = D::KB;
  const int m = s.m, g = s.g;
  const long long id = static_cast<long long>(s.bh) * p.nc + ch;

  // Each part's operands are read while the part before it runs: a wave has its matrix core to itself, and
  // nothing else hides what a read takes. The compiler keeps to the order between sched_barriers.
  f32x4 ks[NC][4], qs[NC][4];
#pragma unroll
  for (int cc = 0; cc < NC; ++cc)
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[cc][i] = qs[cc][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  bf16x8 ka[2][4][NP], qa[2][4][NP], ta[kTriBlocks][3], pa[kTriBlocks][3], vv[NC][2][NP];
#pragma unroll
  for (int i = 0; i < 4; ++i) u.k.rows(i, 0, m, g, ka[0][i]);
  if (!D::KONLY && p.states) s.template store_tiles<0, RT>(p.states, id, delta_tiles(p.dk), S);
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kb + 1 < KB) u.k.rows(i, kb + 1, m, g, ka[(kb + 1) & 1][i]);
      else if constexpr (!D::KONLY) u.q.rows(i, 0, m, g, qa[0][i]);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int cc = 0; cc < NC; ++cc) mma_rows<NP, 3>(ks[cc], ka[kb & 1], sb[cc][kb]);
  }
#pragma unroll
  for (int cc = 0; cc < NC; ++cc)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) u.v.columns(s.w * NC + cc, kb, m, g, vv[cc][kb]);
  const float whole = u.rows[kRowWhole * 64];
  bf16x8 xb[NC][2][3];
  f32x4 y[NC][4];
  float odd = 0.0f;  // not zero where a value read is no number
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    if (!D::KONLY && kb + 1 < KB) {
      if constexpr (!D::KONLY) {
#pragma unroll
        for (int i = 0; i < 4; ++i) u.q.rows(i, kb + 1, m, g, qa[(kb + 1) & 1][i]);
      }
    } else if (!D::KONLY || kb == 0) {
#pragma unroll
      for (int j = 0; j < kTriBlocks; ++j)
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) ta[j][pl] = u.frags[(j * 3 + pl) * 64 + s.lane];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int cc = 0; cc < (D::KONLY ? 0 : NC); ++cc) mma_rows<NP, 3>(qs[cc], qa[kb & 1], sb[cc][kb]);
    if (kb < 2) {  // beside q's products
#pragma unroll
      for (int cc = 0; cc < NC; ++cc) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const f32x4 xg = s.row4(u, kRowX, 2 * kb + i);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            ks[cc][2 * kb + i][r] = fmaf(-xg[r], ks[cc][2 * kb + i][r], plane_sum<NP>(vv[cc][kb], 4 * i + r));
          if (!D::KONLY) {
#pragma unroll
            for (int r = 0; r < 4; ++r) odd = fmaf(ks[cc][2 * kb + i][r], 0.0f, odd);
          }
          y[cc][2 * kb + i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        split_tiles<3>(ks[cc][2 * kb], ks[cc][2 * kb + 1], xb[cc][kb]);
      }
    }
  }
  DeltaBadRows bad[NC];
  const bool apart = !D::KONLY && __builtin_expect(__any(odd != 0.0f), 0);
  if (apart) {
#pragma unroll
    for (int cc = 0; cc < NC; ++cc) bad[cc].take(xb[cc], g);
  }
  __builtin_amdgcn_sched_barrier(0);
  tri_rows<3, 3, NC>(y, ta, xb);
#pragma unroll
  for (int cc = 0; cc < NC; ++cc)
#pragma unroll
    for (int t = 0; t < RT; ++t) S[cc][t] *= whole;  // beside T's products
  if constexpr (!D::KONLY) {
#pragma unroll
    for (int j = 0; j < kTriBlocks; ++j)
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) pa[j][pl] = u.frags[DeltaFrags::T + (j * 3 + pl) * 64 + s.lane];
  }
  constexpr int TG = 2;  // tiles of the state at a time
  bf16x8 yb[NC][2][3], kc[2][TG][2][NP];
#pragma unroll
  for (int t = 0; t < TG; ++t)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) u.k.columns(t, kb, m, g, kc[0][t][kb]);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (!D::KONLY) {  // the output
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 og = s.row4(u, kRowO, i);
#pragma unroll
      for (int cc = 0; cc < NC; ++cc) qs[cc][i] *= og;
    }
#pragma unroll
    for (int cc = 0; cc < NC; ++cc)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) split_tiles<3>(y[cc][2 * kb], y[cc][2 * kb + 1], xb[cc][kb]);
    tri_rows<3, 3, NC>(qs, pa, xb);
    if (apart) {
#pragma unroll
      for (int cc = 0; cc < NC; ++cc) {
        bad[cc].mark(qs[cc], g);
        bad[cc].mark(y[cc], g);
      }
    }
    if (p.ys) s.template store_tiles<0, 4>(p.ys, id, 4, y);
  }
  // the state
#pragma unroll
  for (int cc = 0; cc < NC; ++cc) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[cc][i] *= s.row4(u, kRowS, i);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) split_tiles<3>(y[cc][2 * kb], y[cc][2 * kb + 1], yb[cc][kb]);
  }
#pragma unroll
  for (int t0 = 0; t0 < RT; t0 += TG) {
    if (t0 + TG < RT) {
#pragma unroll
      for (int t = 0; t < TG; ++t)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) u.k.columns(t0 + TG + t, kb, m, g, kc[(t0 / TG + 1) & 1][t][kb]);
      __builtin_amdgcn_sched_barrier(0);
    }
    state_tiles<NP, TG, NC>(S, t0, kc[(t0 / TG) & 1], yb);
#pragma unroll
    for (int t = t0; t < t0 + TG; t += 2)
#pragma unroll
      for (int cc = 0; cc < NC; ++cc) split_tiles<3>(S[cc][t], S[cc][t + 1], sb[cc][t / 2]);
  }
  if constexpr (!D::KONLY) s.result(u, o, ch, qs);
}

template <class UT, int MODE, int DK, int NC, int NW>
__global__ void __launch_bounds__((DeltaScan<UT, MODE, DK, NC, NW, false>::THREADS)) delta_scan_kernel(const DeltaArgs p) {
  typedef DeltaScan<UT, MODE, DK, NC, NW, false> D;
  typedef typename D::Buf Buf;
  constexpr int RT = D::RT, KB = D::KB;
  __shared__ Buf buf[D::NBUF];
  const DeltaView o = {p.o, static_cast<long long>(p.L) * p.HV * p.dv, static_cast<long long>(p.HV) * p.dv};
  D s(p, p.v, 1);
  if (s.idle) return;
  const long long at_state = static_cast<long long>(s.bh) * p.dk * p.dv;
  const int end = s.c0 + s.nch;
  if (s.nch > 0 && (s.loads || !D::NL)) {
    s.fetch(buf[s.c0 & (D::NBUF - 1)]);
    s.land(buf[s.c0 & (D::NBUF - 1)]);
  }
  __syncthreads();
  if (s.loads) {  // every barrier here has its fellow below
    for (int ch = s.c0; ch < end; ++ch) {
      Buf& next = buf[(ch + 1) & (D::NBUF - 1)];
      if (ch > s.c0) s.send(next, o, ch - 1);
      if (ch + 1 < end) {
        s.fetch(next);
        s.land(next);
      }
      __syncthreads();
    }
    if (s.nch > 0) s.send(buf[(end - 1) & (D::NBUF - 1)], o, end - 1);
    return;
  }
  f32x4 S[NC][RT];
  s.join(p.s0 ? p.s0 + at_state : nullptr, S);
  bf16x8 sb[NC][KB][3];
#pragma unroll
  for (int cc = 0; cc < NC; ++cc)
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) split_tiles<3>(S[cc][2 * kb], S[cc][2 * kb + 1], sb[cc][kb]);
  for (int ch = s.c0; ch < end; ++ch) {
    Buf& next = buf[(ch + 1) & (D::NBUF - 1)];
    if (!D::NL && ch + 1 < end) s.fetch(next);
    delta_scan_chunk<D, UT, DK, NC>(s, p, o, ch, buf[ch & (D::NBUF - 1)], S, sb);
    if constexpr (!D::NL) {
      __syncthreads();
      if (ch + 1 < end) s.land(next);
    }
    __syncthreads();
  }
  if (!s.last) return;
  if (p.sT) s.store_state(p.sT + at_state, S);
  // rows behind the last chunk of the sequence
#pragma unroll
  for (int cc = 0; cc < NC; ++cc)
    if (s.col(cc) < p.dv)
      for (long long t = static_cast<long long>(end) * kDeltaChunk + s.g; t < p.L; t += 4)
        store1(out_at<UT>(o, s.b, t) + static_cast<long long>(s.hv) * p.dv + s.col(cc), 0.0f);
}

// A chunk of the adjoint's scan
template <class D, class UT, int DK, int NC>
__device__ __forceinline__ void delta_back_chunk(const D& s, const DeltaArgs& p, const DeltaView& o, int ch, typename D::Buf& u,
                                                 f32x4 (&S)[NC][D::RT], bf16x8 (&sb)[NC][D::KB][3]) {
  constexpr int NP = D::NP, RT = D::RT, KB = D::KB;
  const int m = s.m, g = s.g;
  const long long id = static_cast<long long>(s.bh) * p.nc + ch;

  f32x4 y[NC][4], x[NC][4];
#pragma unroll
  for (int cc = 0; cc < NC; ++cc)
#pragma unroll
    for (int i = 0; i < 4; ++i) y[cc][i] = x[cc][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  bf16x8 ka[2][4][NP], ta[kTriBlocks][3], pa[kTriBlocks][3], vb[NC][2][NP];
#pragma unroll
  for (int i = 0; i < 4; ++i) u.k.rows(i, 0, m, g, ka[0][i]);
  if constexpr (!D::SEGMENT) s.template store_tiles<0, RT>(p.dstates, id, delta_tiles(p.dk), S);
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    if (kb + 1 < KB) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u.k.rows(i, kb + 1, m, g, ka[(kb + 1) & 1][i]);
    } else {
#pragma unroll
      for (int cc = 0; cc < NC; ++cc)
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) u.v.columns(s.w * NC + cc, k2, m, g, vb[cc][k2]);
#pragma unroll
      for (int j = 0; j < kTriBlocks; ++j)
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) pa[j][pl] = u.frags[DeltaFrags::T + (j * 3 + pl) * 64 + s.lane];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int cc = 0; cc < NC; ++cc) mma_rows<NP, 3>(y[cc], ka[kb & 1], sb[cc][kb]);
  }
#pragma unroll
  for (int j = 0; j < kTriBlocks; ++j)
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) ta[j][pl] = u.frags[(j * 3 + pl) * 64 + s.lane];
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x4 sg = s.row4(u, kRowS, i);
#pragma unroll
    for (int cc = 0; cc < NC; ++cc) y[cc][i] *= sg;
  }
  tri_rows<3, NP, NC, true>(y, pa, vb);
  constexpr int TG = NP == 1 ? 2 : 1;  // tiles of the state at a time
  bf16x8 xb[NC][2][3], ob[NC][2][3], kc[2][TG][2][NP], qc[2][TG][2][NP];
#pragma unroll
  for (int cc = 0; cc < NC; ++cc)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) split_tiles<3>(y[cc][2 * kb], y[cc][2 * kb + 1], xb[cc][kb]);
#pragma unroll
  for (int t = 0; t < TG; ++t)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      u.q.columns(t, kb, m, g, qc[0][t][kb]);
      u.k.columns(t, kb, m, g, kc[0][t][kb]);
    }
  __builtin_amdgcn_sched_barrier(0);
  tri_rows<3, 3, NC, true>(x, ta, xb);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x4 og = s.row4(u, kRowO, i);
#pragma unroll
    for (int cc = 0; cc < NC; ++cc)
#pragma unroll
      for (int r = 0; r < 4; ++r) y[cc][i][r] = og[r] * plane_sum<NP>(vb[cc][i / 2], 4 * (i & 1) + r);
  }
  const float whole = u.rows[kRowWhole * 64];
#pragma unroll
  for (int cc = 0; cc < NC; ++cc) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) split_tiles<3>(y[cc][2 * kb], y[cc][2 * kb + 1], ob[cc][kb]);
#pragma unroll
    for (int t = 0; t < RT; ++t) S[cc][t] *= whole;
  }
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (!D::SEGMENT) {
    s.template store_tiles<0, 4>(p.dxs, id, 4, x);
    s.result(u, p.gv, ch, x);
  }
#pragma unroll
  for (int cc = 0; cc < NC; ++cc) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[cc][i] *= -s.row4(u, kRowX, i);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) split_tiles<3>(x[cc][2 * kb], x[cc][2 * kb + 1], xb[cc][kb]);
  }
#pragma unroll
  for (int t0 = 0; t0 < RT; t0 += TG) {
    if (t0 + TG < RT) {
#pragma unroll
      for (int t = 0; t < TG; ++t)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          u.q.columns(t0 + TG + t, kb, m, g, qc[(t0 / TG + 1) & 1][t][kb]);
          u.k.columns(t0 + TG + t, kb, m, g, kc[(t0 / TG + 1) & 1][t][kb]);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    state_tiles<NP, TG, NC>(S, t0, qc[(t0 / TG) & 1], ob);
    state_tiles<NP, TG, NC>(S, t0, kc[(t0 / TG) & 1], xb);
    const int t = t0 + TG - 2;
    if (t >= 0 && t % 2 == 0) {
#pragma unroll
      for (int cc = 0; cc < NC; ++cc) split_tiles<3>(S[cc][t], S[cc][t + 1], sb[cc][t / 2]);
    }
  }
}

// dS from the last chunk to the first; p.s0 is dsT and p.sT is ds0
template <class UT, int MODE, int DK, int NC, int NW>
__global__ void __launch_bounds__((DeltaScan<UT, MODE, DK, NC, NW, true>::THREADS)) delta_back_kernel(const DeltaArgs p) {
  typedef DeltaScan<UT, MODE, DK, NC, NW, true> D;
  typedef typename D::Buf Buf;
  constexpr int RT = D::RT, KB = D::KB;
  __shared__ Buf buf[D::NBUF];
  const DeltaView o = {p.o, static_cast<long long>(p.L) * p.HV * p.dv, static_cast<long long>(p.HV) * p.dv};
  D s(p, o, -1);
  if (s.idle) return;
  const long long at_state = static_cast<long long>(s.bh) * p.dk * p.dv;
  const int end = s.c0 + s.nch;
  if (s.nch > 0 && (s.loads || !D::NL)) {
    s.fetch(buf[(end - 1) & (D::NBUF - 1)]);
    s.land(buf[(end - 1) & (D::NBUF - 1)]);
  }
  __syncthreads();
  if (s.loads) {  // every barrier here has its fellow below
    for (int ch = end - 1; ch >= s.c0; --ch) {
      Buf& next = buf[(ch + 1) & (D::NBUF - 1)];
      if (ch + 1 < end) s.send(next, p.gv, ch + 1);
      if (ch > s.c0) {
        s.fetch(next);
        s.land(next);
      }
      __syncthreads();
    }
    if (s.nch > 0) s.send(buf[s.c0 & (D::NBUF - 1)], p.gv, s.c0);
    return;
  }
  f32x4 S[NC][RT];
  s.join(p.s0 ? p.s0 + at_state : nullptr, S);
  bf16x8 sb[NC][KB][3];
#pragma unroll
  for (int cc = 0; cc < NC; ++cc)
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) split_tiles<3>(S[cc][2 * kb], S[cc][2 * kb + 1], sb[cc][kb]);
  for (int ch = end - 1; ch >= s.c0; --ch) {
    Buf& next = buf[(ch + 1) & (D::NBUF - 1)];
    if (!D::NL && ch > s.c0) s.fetch(next);
    delta_back_chunk<D, UT, DK, NC>(s, p, o, ch, buf[ch & (D::NBUF - 1)], S, sb);
    if constexpr (!D::NL) {
      __syncthreads();
      if (ch > s.c0) s.land(next);
    }
    __syncthreads();
  }
  if (p.sT && s.seg == 0) s.store_state(p.sT + at_state, S);
  if (!s.last) return;
  // rows behind the last chunk of the sequence
#pragma unroll
  for (int cc = 0; cc < NC; ++cc)
    if (s.col(cc) < p.dv)
      for (long long t = static_cast<long long>(end) * kDeltaChunk + s.g; t < p.L; t += 4)
        store1(out_at<UT>(p.gv, s.b, t) + static_cast<long long>(s.hv) * p.dv + s.col(cc), 0.0f);
}

// What each segment makes of the state in front of it (ADJ: of dS behind it)
template <class UT, int MODE, int DK, int NC, int NW, bool ADJ>
__global__ void __launch_bounds__((DeltaScan<UT, MODE, DK, NC, NW, ADJ, true>::THREADS)) delta_segment_kernel(const DeltaArgs p) {
  typedef DeltaScan<UT, MODE, DK, NC, NW, ADJ, true> D;
  typedef typename D::Buf Buf;
  constexpr int RT = D::RT, KB = D::KB, DIR = ADJ ? -1 : 1;
  __shared__ Buf buf[D::NBUF];
  const DeltaView o = {p.o, static_cast<long long>(p.L) * p.HV * p.dv, static_cast<long long>(p.HV) * p.dv};
  D s(p, ADJ ? o : p.v, DIR);
  if (s.idle) return;  // else there are chunks
  const int first = ADJ ? s.c0 + s.nch - 1 : s.c0, end = ADJ ? s.c0 - 1 : s.c0 + s.nch;
  if (s.loads || !D::NL) {
    s.fetch(buf[first & (D::NBUF - 1)]);
    s.land(buf[first & (D::NBUF - 1)]);
  }
  __syncthreads();
  if (s.loads) {  // every barrier here has its fellow below
    for (int ch = first; ch != end; ch += DIR) {
      Buf& next = buf[(ch + 1) & (D::NBUF - 1)];
      if (ch + DIR != end) {
        s.fetch(next);
        s.land(next);
      }
      __syncthreads();
    }
    return;
  }
  f32x4 S[NC][RT];
  if (s.ident) s.identity(S);
  else s.load_state(p.s0 && (ADJ ? s.last : s.seg == 0) ? p.s0 + static_cast<long long>(s.bh) * p.dk * p.dv : nullptr, S);
  bf16x8 sb[NC][KB][3];
#pragma unroll
  for (int cc = 0; cc < NC; ++cc)
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) split_tiles<3>(S[cc][2 * kb], S[cc][2 * kb + 1], sb[cc][kb]);
  for (int ch = first; ch != end; ch += DIR) {
    Buf& next = buf[(ch + 1) & (D::NBUF - 1)];
    if (!D::NL && ch + DIR != end) s.fetch(next);
    if constexpr (ADJ) delta_back_chunk<D, UT, DK, NC>(s, p, o, ch, buf[ch & (D::NBUF - 1)], S, sb);
    else delta_scan_chunk<D, UT, DK, NC>(s, p, o, ch, buf[ch & (D::NBUF - 1)], S, sb);
    if constexpr (!D::NL) {
      __syncthreads();
      if (ch + DIR != end) s.land(next);
    }
    __syncthreads();
  }
  s.store_segment(S);
}

// A workgroup per chunk and head of q and k: the gradients of q, k, v and the
// gates. Wave (i, f): the chunk's 16 rows i, columns f of two halves of dk. dv goes
// by in blocks of 32 columns, two of them on their way in registers. B = 8 L = 4096
// H = 8, 128 wide, bf16: 480 to 510 us for 1170 MB of states, dS, y, dX, inputs and
// gradients (2.4 TB/s). One workgroup fits a CU (118 KB), so its parts follow each
// other: of 57000 cycles 20000 are waits for loads, 10000 the products over dv, 22000
// the rest, most of it reads of workgroup memory (4700 of them, a seventh more for
// banks that collide).
template <class UT, int DK>
struct DeltaGradLds {
  static constexpr int NP = DeltaPlanes<UT>::NP, RT = DK / 16;
  typedef DeltaTile<DK, NP> Tile;
  struct Stage {  // 32 columns of dv, which are the rows of all but dO
    DeltaTile<DK, 3, 32> s, ds;
    DeltaTile<64, 3, 32> y, x;
    DeltaTile<32, NP> o;
  };
  static constexpr bool APART = sizeof(Stage) + 2 * sizeof(Tile) <= 120 * 1024;  // the tiles beside the stage
  static constexpr int ROW = 68;
  struct Mats { float d0[64 * ROW], d1[64 * ROW], w[64 * ROW]; };
  static constexpr size_t a16(size_t x) { return (x + 15) / 16 * 16; }
  // stage | (d0, d1 on the stage where the tiles lie apart, else behind the tiles)
  static constexpr size_t kStage = a16(sizeof(Stage)), kTiles = a16(2 * sizeof(Tile));
  static constexpr size_t TILES = APART ? kStage : 0;
  static constexpr size_t MATS = APART ? 0 : kTiles;
  static constexpr size_t BYTES = APART ? kStage + kTiles : (kStage > kTiles + sizeof(Mats) ? kStage : kTiles + sizeof(Mats));
};

// SHARED: several value heads to a head of q and k, whose gradients are summed over them
template <class UT, bool EVEN, int DK, bool SHARED>
__global__ void __launch_bounds__(512) delta_grad_kernel(const DeltaArgs p) {
  typedef DeltaGradLds<UT, DK> M;
  typedef typename M::Tile Tile;
  constexpr int NP = M::NP, RT = M::RT, HT = RT / 2, ROW = M::ROW;
  static_assert(M::BYTES + 10240 <= 160 * 1024, "fits the workgroup's memory");
  static_assert(sizeof(typename M::Mats) <= M::kStage || !M::APART, "the matrices fit where the stage was");
  __shared__ __attribute__((aligned(16))) char lds[M::BYTES];
  __shared__ float srow[kRows * 64], spart[2][5][64], sdot[8], scol[8][64], spass[64];
  typename M::Stage& sg = *reinterpret_cast<typename M::Stage*>(lds);
  Tile& tk = reinterpret_cast<Tile*>(lds + M::TILES)[0];
  Tile& tq = reinterpret_cast<Tile*>(lds + M::TILES)[1];
  typename M::Mats& mt = *reinterpret_cast<typename M::Mats*>(lds + M::MATS);

  const int tid = threadIdx.x, lane = tid & 63, w8 = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int w = w8 & 3, f = w8 >> 2, per = SHARED ? p.HV / p.H : 1;
  const int ch = blockIdx.x % p.nc, b = blockIdx.x / p.nc / p.H, h = blockIdx.x / p.nc % p.H;
  const int t0 = ch * kDeltaChunk, len = delta_len(p, b), rows_out = min(p.L - t0, kDeltaChunk);
  if (t0 >= len) {  // no step: zeros
    for (int i = tid; i < rows_out * p.dk; i += 512) {
      store1(out_at<UT>(p.gq, b, t0 + i / p.dk) + h * p.dk + i % p.dk, 0.0f);
      store1(out_at<UT>(p.gk, b, t0 + i / p.dk) + h * p.dk + i % p.dk, 0.0f);
    }
    for (int i = tid; i < rows_out * per; i += 512) {
      UT* to = out_at<UT>(p.dgates, b, t0 + i / per) + h * per + i % per;
      store1(to, 0.0f);
      store1(to + p.HV, 0.0f);
    }
    for (int i = tid; i < (p.dlam_part ? per : 0); i += 512)
      p.dlam_part[(static_cast<long long>(h) * per + i) * p.B * p.nc + b * p.nc + ch] = 0.0f;
    return;
  }
  const int n = min(len - t0, kDeltaChunk);
  constexpr float kLog2e = 1.4426950408889634f;
  auto tiles = [&]() {
    constexpr int N = (64 * DK / 8 + 511) / 512;
    const __amdgpu_buffer_rsrc_t kr = rows_of<UT>(p.k, b, t0, h * p.dk, n, p.H * p.dk);
    const __amdgpu_buffer_rsrc_t qr = rows_of<UT>(p.q, b, t0, h * p.dk, n, p.H * p.dk);
    Piece<UT, EVEN> a[N], c[N];
    const int row = tid / (DK / 8), d = Tile::source(tid);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = row + 512 / (DK / 8) * i;
      a[i].load(kr, offset_of<UT>(r, p.k.token, d, r < n && d < p.dk));
      c[i].load(qr, offset_of<UT>(r, p.q.token, d, r < n && d < p.dk));
    }
    bf16x8 o[NP];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      planes_of(a[i], p.dk - d, o);
      tk.put_slot(tid + 512 * i, o);
      planes_of(c[i], p.dk - d, o);
      tq.put_slot(tid + 512 * i, o);
    }
  };
  if constexpr (M::APART) tiles();

  f32x4 dq[SHARED ? HT : 1], dk[SHARED ? HT : 1];
  float qsum[SHARED ? 4 : 1], ksum[SHARED ? 4 : 1];  // q.dQ and k.dK over the value heads, of the lane's 4 rows
  if constexpr (SHARED) {
#pragma unroll
    for (int t = 0; t < HT; ++t) dq[t] = dk[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < 4; ++r) qsum[r] = ksum[r] = 0.0f;
  }
  for (int hr = 0; hr < per; ++hr) {
    // made anew in every round, so that no address is held over the rounds
    int m = lane & 15, g = lane >> 4;
    __asm__ volatile("" : "+v"(m), "+v"(g));
    // the lane's 4 rows of column m of a tile of q or k, from the operand that holds them
    auto mine = [&](Tile& t, int tile, float (&v)[4]) {
      bf16x8 o[NP];
      t.columns(f * HT + tile, w >> 1, m, g, o);
  #pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = w & 1 ? plane_sum<NP>(o, 4 + r) : plane_sum<NP>(o, r);
    };
    const int hv = h * per + hr;
    const long long id = (static_cast<long long>(b) * p.HV + hv) * p.nc + ch;
    const int rt = delta_tiles(p.dk), nct = delta_tiles(p.dv);
    const DeltaView ov = {p.o, static_cast<long long>(p.L) * p.HV * p.dv, static_cast<long long>(p.HV) * p.dv};
    const __amdgpu_buffer_rsrc_t orr = rows_of<UT>(ov, b, t0, hv * p.dv, n, p.HV * p.dv);
    // all that a chunk has lies in one run of memory: 32-bit offsets
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(p.states + id * nct * rt * 64, nct * rt * 1024),
                                 dsr = make_rsrc(p.dstates + id * nct * rt * 64, nct * rt * 1024),
                                 yr = make_rsrc(p.ys + id * nct * 4 * 64, nct * 4096),
                                 xr = make_rsrc(p.dxs + id * nct * 4 * 64, nct * 4096);
    // the thread's share of a block of 32 columns, ahead of its use: waves deal out the tiles
    constexpr int NS = RT * 2 / 8;
    constexpr int AHEAD = NP == 1 && (DK == 64 || !SHARED) ? 2 : 1;  // blocks on their way, by the registers that are left
    i32x4 fs[AHEAD][NS], fd[AHEAD][NS], fy[AHEAD], fx[AHEAD];
    Piece<UT, EVEN> fo[AHEAD];
    auto fetch = [&](int vb, auto zc) __attribute__((always_inline)) {
      constexpr int z = decltype(zc)::value;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int e = w8 + 8 * i, c = 2 * vb + e / RT, t = e % RT;
        const uint32_t off = t < rt ? static_cast<uint32_t>((c * rt + t) * 64 + lane) * 16 : kNoLoad;
        fs[z][i] = __builtin_amdgcn_raw_buffer_load_b128(sr, off, 0, 0);
        fd[z][i] = __builtin_amdgcn_raw_buffer_load_b128(dsr, off, 0, 0);
      }
      const uint32_t off = static_cast<uint32_t>(((2 * vb + f) * 4 + w) * 64 + lane) * 16;
      fy[z] = __builtin_amdgcn_raw_buffer_load_b128(yr, off, 0, 0);
      fx[z] = __builtin_amdgcn_raw_buffer_load_b128(xr, off, 0, 0);
      const int row = tid >> 2, d = 32 * vb + sg.o.source(tid);
      if (f == 0) fo[z].load(orr, offset_of<UT>(row, ov.token, d, row < n && d < p.dv));
    };
    typedef std::integral_constant<int, 0> Z0;
    typedef std::integral_constant<int, AHEAD - 1> Z1;
    fetch(0, Z0{});
    if (AHEAD == 2) fetch(1, Z1{});  // past the last block: zeros
    for (int i = tid; i < kRows * 64; i += 512) srow[i] = p.rows[id * (kRows * 64) + i];
    f32x4 qo[HT], kx[HT], yd[HT], dd[4];
    float dot = 0.0f;
#pragma unroll
    for (int t = 0; t < HT; ++t) qo[t] = kx[t] = yd[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j) dd[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int nb = (p.dv + 31) / 32;
    auto block = [&](int vb, auto zc) __attribute__((always_inline)) {
      constexpr int z = decltype(zc)::value;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int e = w8 + 8 * i, c = e / RT, t = e % RT;
        const f32x4 a = __builtin_bit_cast(f32x4, fs[z][i]), d = __builtin_bit_cast(f32x4, fd[z][i]);
#pragma unroll
        for (int r = 0; r < 4; ++r) dot = fmaf(a[r], d[r], dot);
        sg.s.put4(16 * c + m, delta_label(t, 4 * g), a);
        sg.ds.put4(16 * c + m, delta_label(t, 4 * g), d);
      }
      sg.y.put4(16 * f + m, delta_label(w, 4 * g), __builtin_bit_cast(f32x4, fy[z]));
      sg.x.put4(16 * f + m, delta_label(w, 4 * g), __builtin_bit_cast(f32x4, fx[z]));
      if (f == 0) {
        bf16x8 o[NP];
        planes_of(fo[z], p.dv - 32 * vb - sg.o.source(tid), o);
        sg.o.put_slot(tid, o);
      }
      __syncthreads();
      if (vb + AHEAD < nb) fetch(vb + AHEAD, zc);
      bf16x8 ao[NP], ax[3], ay[3], bs[2][3], bd[2][3];
      sg.o.rows(w, 0, m, g, ao);
      sg.x.columns(w, 0, m, g, ax);
      sg.y.columns(w, 0, m, g, ay);
      sg.s.columns(f * HT, 0, m, g, bs[0]);
      sg.ds.columns(f * HT, 0, m, g, bd[0]);
#pragma unroll
      for (int t = 0; t < HT; ++t) {  // the next tile's operands under this one's products
        if (t + 1 < HT) {
          sg.s.columns(f * HT + t + 1, 0, m, g, bs[(t + 1) & 1]);
          sg.ds.columns(f * HT + t + 1, 0, m, g, bd[(t + 1) & 1]);
        } else {
          sg.y.columns(0, 0, m, g, bs[(t + 1) & 1]);
        }
        __builtin_amdgcn_sched_barrier(0);
        const bf16x8(&u)[3] = bs[t & 1], (&v)[3] = bd[t & 1];
#pragma unroll
        for (int q = 2; q >= 0; --q)
#pragma unroll
          for (int i = 0; i <= q; ++i) {
            kx[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ax[i], u[q - i], kx[t], 0, 0, 0);
            yd[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ay[i], v[q - i], yd[t], 0, 0, 0);
            if (i < NP) qo[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ao[i], u[q - i], qo[t], 0, 0, 0);
          }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
          if (j < w) sg.y.columns(j + 1, 0, m, g, bs[(HT + j + 1) & 1]);
          __builtin_amdgcn_sched_barrier(0);
          if (f == 0) mma<NP, 3>(dd[j], ao, bs[(HT + j) & 1]);
          else mma<3, 3>(dd[j], ax, bs[(HT + j) & 1]);
        }
    };
    for (int vb = 0; vb < nb; vb += AHEAD) {
      block(vb, Z0{});
      if (AHEAD == 2 && vb + 1 < nb) block(vb + 1, Z1{});
    }
    __syncthreads();  // the stage has been read
    if constexpr (!M::APART) tiles();
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) dot += __shfl_xor(dot, off, 64);
    if (lane == 0) sdot[w8] = dot;
    if constexpr (!M::APART) __syncthreads();
    // D0 and D1, and W of the one and the other half of the waves
    float* to = f ? mt.d1 : mt.d0;
    f32x4 pp[4];  // q.k, or k.k
#pragma unroll
    for (int j = 0; j < 4; ++j) pp[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kb = 0; kb < DK / 32; ++kb) {
      bf16x8 a[NP], c[NP];
      if (f) tk.rows(w, kb, m, g, a);
      else tq.rows(w, kb, m, g, a);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
          tk.rows(j, kb, m, g, c);
          mma<NP, NP>(pp[j], a, c);
        }
    }
    {
      const f32x4 Gi = *reinterpret_cast<const f32x4*>(&srow[kRowG * 64 + 16 * w + 4 * g]);
      const f32x4 Li = *reinterpret_cast<const f32x4*>(&srow[kRowGLow * 64 + 16 * w + 4 * g]);
      const f32x4 si = *reinterpret_cast<const f32x4*>(&srow[kRowSeg * 64 + 16 * w + 4 * g]);
      const f32x4 li = *reinterpret_cast<const f32x4*>(&srow[(f ? kRowK : kRowQ) * 64 + 16 * w + 4 * g]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = 16 * j + m;
        float* const at = to + (16 * w + 4 * g) * ROW + c;
        if (j > w) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            at[e * ROW] = 0.0f;
            if (!f) mt.w[(16 * w + 4 * g + e) * ROW + c] = 0.0f;
          }
          continue;
        }
        const float Gc = srow[kRowG * 64 + c], sc = srow[kRowSeg * 64 + c], kc = srow[kRowK * 64 + c];
        const f32x4 gap = log_gap(Gi, Li, Gc, srow[kRowGLow * 64 + c]);
        const float bc = (f ? -1.0f : p.scale) * srow[kRowB * 64 + c];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 16 * w + 4 * g + e;
          const bool low = (f ? i > c : i >= c) && si[e] == sc;
          const float d = low ? bc * __builtin_amdgcn_exp2f(gap[e] * kLog2e) * dd[j][e] : 0.0f;
          at[e * ROW] = d;
          pp[j][e] *= d * li[e] * kc;
          if (!f) mt.w[i * ROW + c] = pp[j][e];
        }
      }
    }
    __syncthreads();
    if (f) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
#pragma unroll
          for (int e = 0; e < 4; ++e) mt.w[(16 * w + 4 * g + e) * ROW + 16 * j + m] += pp[j][e];
        }
    }
    const float se = srow[kRowSeg * 64 + 63], Ge = srow[kRowG * 64 + 63], Le = srow[kRowGLow * 64 + 63];
    const f32x4 rq = *reinterpret_cast<const f32x4*>(&srow[kRowQ * 64 + 16 * w + 4 * g]);
    const f32x4 rk = *reinterpret_cast<const f32x4*>(&srow[kRowK * 64 + 16 * w + 4 * g]);
    float part[5][4];  // q.dQ, k.(dK read), k.(dK written); of S1, from S0
    {
      float cq[4], ck[4], cw[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * w + 4 * g + r;
        const float G = srow[kRowG * 64 + i], seg = srow[kRowSeg * 64 + i];
        ck[r] = seg == 0.0f ? -__builtin_amdgcn_exp2f(G * kLog2e) : 0.0f;
        cq[r] = -p.scale * ck[r];
        const float rest = log_gap(Ge, Le, G, srow[kRowGLow * 64 + i]);
        cw[r] = seg == se ? __builtin_amdgcn_exp2f(rest * kLog2e) * srow[kRowB * 64 + i] : 0.0f;
        part[0][r] = part[1][r] = part[2][r] = part[3][r] = part[4][r] = 0.0f;
      }
#pragma unroll
      for (int t = 0; t < HT; ++t) {  // what the states bring: kx and yd become the two parts of dK
        float qv[4], kv[4];
        mine(tq, t, qv);
        mine(tk, t, kv);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          qo[t][r] *= cq[r];
          kx[t][r] *= ck[r];
          yd[t][r] *= cw[r];
          part[3][r] = fmaf(yd[t][r], rk[r] * kv[r], part[3][r]);
          part[4][r] = fmaf(kx[t][r], rk[r] * kv[r], fmaf(qo[t][r], rq[r] * qv[r], part[4][r]));
        }
      }
    }
    // rows (COLS false) or columns of a matrix, block kb of 32 inner indexes, times a factor of those
    auto operand = [&](const float* mat, bool cols, int kind, int kb, bf16x8 (&o)[3]) {
      float x[8];
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        const int c = 32 * kb + 16 * h2 + 4 * g, r = 16 * w + m;
        const f32x4 fc = *reinterpret_cast<const f32x4*>(&srow[kind * 64 + c]);
        f32x4 v;
        if (cols) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = mat[(c + e) * ROW + r];
        } else {
          v = *reinterpret_cast<const f32x4*>(&mat[r * ROW + c]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * h2 + e] = v[e] * fc[e];
      }
      split8<3>(x, o);
    };
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      bf16x8 ca[3], cb[3];
      if (kb <= w / 2) {  // rows of D0 and D1 on k
        operand(mt.d0, false, kRowK, kb, ca);
        operand(mt.d1, false, kRowK, kb, cb);
#pragma unroll
        for (int t = 0; t < HT; ++t) {
          bf16x8 o[NP];
          tk.columns(f * HT + t, kb, m, g, o);
          mma<3, NP>(qo[t], ca, o);
          mma<3, NP>(kx[t], cb, o);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (kb >= w / 2) {  // their columns on q and k
        operand(mt.d0, true, kRowQ, kb, ca);
        operand(mt.d1, true, kRowK, kb, cb);
#pragma unroll
        for (int t = 0; t < HT; ++t) {
          bf16x8 o[NP], o2[NP];
          tq.columns(f * HT + t, kb, m, g, o);
          tk.columns(f * HT + t, kb, m, g, o2);
          mma<3, NP>(yd[t], ca, o);
          mma<3, NP>(yd[t], cb, o2);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int t = 0; t < HT; ++t) {
      float qv[4], kv[4];
      mine(tq, t, qv);
      mine(tk, t, kv);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        part[0][r] = fmaf(rq[r] * qv[r], qo[t][r], part[0][r]);
        part[1][r] = fmaf(rk[r] * kv[r], kx[t][r], part[1][r]);
        part[2][r] = fmaf(rk[r] * kv[r], yd[t][r], part[2][r]);
      }
      if constexpr (SHARED) {
        dq[t] += qo[t];
        dk[t] += kx[t] + yd[t];
      }
    }
    {  // over the 16 lanes of a row: lane m ends up with kind m / 4 of row 4 g + m % 4, and with the fifth kind's
      float v[16], u[4];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = part[i >> 2][i & 3];
#pragma unroll
      for (int r = 0; r < 4; ++r) u[r] = part[4][r];
      sum_and_deal<16, 16>(v, lane);
      sum_and_deal<4, 16>(u, lane);
      spart[f][m >> 2][16 * w + 4 * g + (m & 3)] = v[0];
      if ((m & 3) == 0) spart[f][4][16 * w + 4 * g + (m >> 2)] = u[0];
    }
    __syncthreads();  // W has both halves' part: its rows are summed by other waves than those that added to it
    // sums of W over j < t <= i: a wave takes 8 t, a lane a column j
    {
      float v = 0.0f;
#pragma unroll
      for (int r = 0; r < 8; ++r) v += mt.w[(8 * w8 + r) * ROW + lane];
      scol[w8][lane] = v;
    }
    __syncthreads();
    {
      float v = 0.0f, pass[8];
      for (int k = 7; k > w8; --k) v += scol[k][lane];
#pragma unroll
      for (int r = 7; r >= 0; --r) {
        v += mt.w[(8 * w8 + r) * ROW + lane];
        pass[r] = lane < 8 * w8 + r ? v : 0.0f;
      }
      sum_and_deal<8, 64>(pass, lane);
      if ((lane & 7) == 0) spass[8 * w8 + deal_index<8, 64>(lane)] = pass[0];
    }
    if constexpr (SHARED) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * w + 4 * g + r;
        qsum[r] += spart[0][0][i] + spart[1][0][i];
        ksum[r] += spart[0][1][i] + spart[1][1][i] + spart[0][2][i] + spart[1][2][i];
      }
    }
    // Gradients through the lengths of q and k: r (d - unit (unit.d))
    auto finish = [&]() {
      float qs[4], ks[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * w + 4 * g + r;
        if constexpr (SHARED) {
          qs[r] = qsum[r];
          ks[r] = ksum[r];
        } else {
          qs[r] = spart[0][0][i] + spart[1][0][i];
          ks[r] = spart[0][1][i] + spart[1][1][i] + spart[0][2][i] + spart[1][2][i];
        }
      }
      // two tiles are 8 neighbouring columns of 4 lanes' rows: transposed within those lanes, a lane has 8
      // columns of its row m % 4
      const int row = 16 * w + 4 * g + (m & 3);
      UT* const qo_ = out_at<UT>(p.gq, b, t0 + row) + h * p.dk;
      UT* const ko_ = out_at<UT>(p.gk, b, t0 + row) + h * p.dk;
#pragma unroll
      for (int t = 0; t < HT; t += 2) {
        float oq[8], ok[8];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float qv[4], kv[4], vq[4], vk[4];
          mine(tq, t + z, qv);
          mine(tk, t + z, kv);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float a, c;
            if constexpr (SHARED) {
              a = dq[t + z][r];
              c = dk[t + z][r];
            } else {
              a = qo[t + z][r];
              c = kx[t + z][r] + yd[t + z][r];
            }
            const bool live = 16 * w + 4 * g + r < n;  // else zero, whatever the other rows are
            vq[r] = live ? rq[r] * fmaf(-rq[r] * qv[r], qs[r], a) : 0.0f;
            vk[r] = live ? rk[r] * fmaf(-rk[r] * kv[r], ks[r], c) : 0.0f;
          }
          transpose4(vq, lane);
          transpose4(vk, lane);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            oq[4 * z + c] = vq[c];
            ok[4 * z + c] = vk[c];
          }
        }
        const int d = 16 * f * HT + 16 * t + 8 * (m >> 2), count = p.dk - d;
        if (row < rows_out && count > 0) {
          store_run(qo_ + d, oq, count, p.wide_qk);
          store_run(ko_ + d, ok, count, p.wide_qk);
        }
      }
    };
    if (!SHARED || hr + 1 == per) finish();
    __syncthreads();
    if (w8 == 0) {  // the gates: a lane per step
      const int i = lane;
      const float bw = spart[0][2][i] + spart[1][2][i], to_s1 = spart[0][3][i] + spart[1][3][i];
      float from = spart[0][4][i] + spart[1][4][i], into = to_s1;
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss += sdot[k];
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const float u = __shfl_down(from, o, 64), v = __shfl_up(into, o, 64);
        if (i + o < 64) from += u;  // over this row and later ones
        if (i >= o) into += v;
      }
      into = __shfl_up(into, 1, 64);  // over the rows in front of this one
      const float G = spass[i] + from + (i > 0 ? into : 0.0f) + srow[kRowWhole * 64] * ss;
      const float dl = i < n ? G : 0.0f;
      const float r = srow[kRowR * 64 + i], lam = p.lam[hv];
      if (i < rows_out) {
        UT* go = out_at<UT>(p.dgates, b, t0 + i) + hv;
        store1(go, i < n ? -p.c * softplus(lam) * dl * r * srow[kRowNotR * 64 + i] : 0.0f);
        store1(go + p.HV, i < n ? bw * srow[kRowNotB * 64 + i] : 0.0f);
      }
      if (p.dlam_part) {
        float sum = dl * r;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
        if (i == 0) p.dlam_part[static_cast<long long>(hv) * p.B * p.nc + b * p.nc + ch] = sum;
      }
    }
    if (SHARED && hr + 1 < per) __syncthreads();
  }
}

// dlam[hv] = -c s(lam) sum of its chunks' parts, in a fixed order
__global__ void __launch_bounds__(256) delta_dlam_kernel(const float* part, const float* lam, float* dlam, int n, float c) {
  __shared__ float s[256];
  const int hv = blockIdx.x, tid = threadIdx.x;
  float v = 0.0f;
  for (int i = tid; i < n; i += 256) v += part[static_cast<long long>(hv) * n + i];
  s[tid] = v;
  __syncthreads();
#pragma unroll
  for (int o = 128; o >= 1; o >>= 1) {
    if (tid < o) s[tid] += s[tid + o];
    __syncthreads();
  }
  if (tid == 0) dlam[hv] = -c * sigm(lam[hv]) * s[0];
}

struct DeltaStepArgs {
  const void *q, *k, *v, *gates;        // rows of a request, `*_row` elements apart
  long long q_row, k_row, v_row, g_row;
  const float* lam;
  const int* slots;
  float* state;  // [S][HV][dk][dv]
  void* o;       // [B][HV][dv]
  int B, H, HV, dk, dv, S;
  float c, eps, scale;
  int wide;      // rows of the state take 16-byte accesses
};

// One token: a workgroup per request, value head and 32 columns of the state,
// 4 columns and every 32nd row per thread. o = a S^T q + (q.k) u needs the old
// state only, so both sums over the rows come from one pass, and the state is read
// and written once. 64 requests of 32 heads of 128 x 128: 53 to 57 us, 4.7 to 5.1 TB/s, what a copy
// reaches; one request of 8 heads: 5.5 us, the latency of two dependent loads and a launch.
template <class UT>
__global__ void __launch_bounds__(256) delta_step_kernel(const DeltaStepArgs p) {
  constexpr int NR = 4;  // rows per thread: dk <= 128
  __shared__ float sq[128], sk[128];
  __shared__ f32x4 sum[4][2][8];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int nsl = (p.dv + 31) / 32;
  const int sl = blockIdx.x % nsl, bh = blockIdx.x / nsl, b = bh / p.HV, hv = bh % p.HV, h = hv / (p.HV / p.H);
  const int cg = tid & 7, r0 = tid >> 3, col = 32 * sl + 4 * cg;
  const int slot = p.slots ? p.slots[b] : b;
  UT* out = static_cast<UT*>(p.o) + (static_cast<long long>(b) * p.HV + hv) * p.dv;
  if (slot < 0 || slot >= p.S) {  // no request
    if (tid < 32 && 32 * sl + tid < p.dv) store1(out + 32 * sl + tid, 0.0f);
    return;
  }
  float* S = p.state + (static_cast<long long>(slot) * p.HV + hv) * p.dk * p.dv;
  f32x4 s[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = r0 + 32 * i;
    s[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (r < p.dk) {
      const float* at = S + static_cast<long long>(r) * p.dv + col;
      if (p.wide) {
        if (col < p.dv) s[i] = *reinterpret_cast<const f32x4*>(at);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < p.dv) s[i][e] = at[e];
      }
    }
  }
  const UT* q = static_cast<const UT*>(p.q) + b * p.q_row + h * p.dk;
  const UT* k = static_cast<const UT*>(p.k) + b * p.k_row + h * p.dk;
  const UT* gp = static_cast<const UT*>(p.gates) + b * p.g_row + hv;
  float qv[2], kv[2], sums[3] = {0.0f, 0.0f, 0.0f};  // q.q, k.k, q.k; every wave has them all
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int d = lane + 64 * i;
    qv[i] = d < p.dk ? load1(q + d) : 0.0f;
    kv[i] = d < p.dk ? load1(k + d) : 0.0f;
    sums[0] = fmaf(qv[i], qv[i], sums[0]);
    sums[1] = fmaf(kv[i], kv[i], sums[1]);
    sums[2] = fmaf(qv[i], kv[i], sums[2]);
  }
  const float a = __builtin_amdgcn_exp2f(-p.c * softplus(p.lam[hv]) * sigm(load1(gp)) * 1.4426950408889634f);
  const float beta = sigm(load1(gp + p.HV));
  float vv[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    vv[e] = col + e < p.dv ? load1(static_cast<const UT*>(p.v) + b * p.v_row + static_cast<long long>(hv) * p.dv + col + e) : 0.0f;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1)
#pragma unroll
    for (int j = 0; j < 3; ++j) sums[j] += __shfl_xor(sums[j], off, 64);
  const float rq = 1.0f / sqrtf(sums[0] + p.eps), rk = 1.0f / sqrtf(sums[1] + p.eps);
  if (w == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sq[lane + 64 * i] = qv[i] * rq;
      sk[lane + 64 * i] = kv[i] * rk;
    }
  }
  __syncthreads();
  f32x4 ps = {0.0f, 0.0f, 0.0f, 0.0f}, os = ps;
  float kr[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const float x = sq[r0 + 32 * i];
    kr[i] = sk[r0 + 32 * i];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ps[e] = fmaf(kr[i], s[i][e], ps[e]);
      os[e] = fmaf(x, s[i][e], os[e]);
    }
  }
#pragma unroll
  for (int off = 8; off <= 32; off <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ps[e] += __shfl_xor(ps[e], off, 64);
      os[e] += __shfl_xor(os[e], off, 64);
    }
  if (lane < 8) {
    sum[w][0][lane] = ps;
    sum[w][1][lane] = os;
  }
  __syncthreads();
  ps = sum[0][0][cg] + sum[1][0][cg] + sum[2][0][cg] + sum[3][0][cg];
  os = sum[0][1][cg] + sum[1][1][cg] + sum[2][1][cg] + sum[3][1][cg];
  f32x4 u;
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = beta * fmaf(-a, ps[e], vv[e]);
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = r0 + 32 * i;
    if (r < p.dk) {
      f32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = fmaf(kr[i], u[e], a * s[i][e]);
      float* at = S + static_cast<long long>(r) * p.dv + col;
      if (p.wide) {
        if (col < p.dv) *reinterpret_cast<f32x4*>(at) = x;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < p.dv) at[e] = x[e];
      }
    }
  }
  if (r0 == 0) {
    const float qk = sums[2] * rq * rk;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < p.dv) store1(out + col + e, p.scale * fmaf(a, os[e], qk * u[e]));
  }
}

}  // namespace pararnn
