// matmul_fp8.h -- product of two 8-bit (e4m3) matrices with a scale for each
// block of 128 along K:
//   y[m][n] = sum_k a[m][k] sa[k / 128][m] w[n][k] sw[n / rows][k / 128] + bias[n],
// rows = 128 (a scale per 128 x 128 block of w) or 1 (one per row).
//
// A wave holds 16 x 16 tiles of y^T: w is the matrix instruction's first
// operand, so that a lane ends up with 4 consecutive columns of one row of y,
// and one fp32 scale of a covers them. Both operands take their 32 bytes of a
// 128-block per lane in the same order, so any order does.
//
// The 8-bit matrix instructions add their products eight at a time (k in
// order), each cut toward zero to a multiple of 2^-13 of the power of two of the
// largest of the eight; the sums of eight, and the running sum where the
// instruction carries it (e8m0 scales), are added in fp32 (measured in the
// 16x16x128 form that is used here). A result is so off by at most 7 x 2^-13 =
// 2^-10.2 of the sum of its products' magnitudes. Measured, of that sum, at K =
// 128 and 4096: Gaussian operands 2.2e-6 and 3.7e-7 root mean square, 1.2e-5 and
// 1.5e-6 at most; operands spread over many powers of two (Gaussian times exp of
// twice a Gaussian) 3.5e-5 and 1.6e-5, 2.4e-4 and 1e-4 at most; positive ones of
// one size 4e-7 to 1e-6, over 2^20 products as over 2^12. A bf16 result takes
// it: for Gaussian operands it is a hundredth of the result's own rounding (root
// mean square) and turns one in five hundred of them; it exceeds that rounding
// where products over many powers of two cancel. An fp32 result keeps its
// digits: its operands are widened to bf16, which holds every e4m3 value, and
// multiplied in that type, whose sums are good to 1e-8.
// The product of two scales is formed in fp32 in all but the e8m0 tiles: scales
// that multiply to less than 2^-126 lose digits, to 2^128 or more are infinite.
#pragma once

#include <type_traits>

#include "layer_common.h"

namespace pararnn {

struct MatmulArgs {
  const uint8_t* a;   // [M][K]
  const void* sa;     // [KB][M], fp32 or e8m0
  const uint8_t* w;   // [N][K]
  const void* sw;     // [ceil(N / rows)][KB]
  const float* bias;  // [N] or nullptr
  void* y;            // [M][N] bf16 or fp32
  int M, N, K, KB;
  int vec;            // columns of y that go out at a time, by the alignment of y and its rows: 8, 4 or 1
  int stream;         // y is larger than the last-level cache
};

// 4 columns of y at element i, `left` of them inside the row
template <bool F32OUT>
__device__ __forceinline__ void store_row4(void* y, long long i, int left, int vec, const float (&o)[4]) {
  if constexpr (F32OUT) {
    float* q = static_cast<float*>(y) + i;
    if (vec >= 4) {
      *reinterpret_cast<f32x4*>(q) = f32x4{o[0], o[1], o[2], o[3]};
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (v < left) q[v] = o[v];
    }
  } else {
    bf16* q = static_cast<bf16*>(y) + i;
    const uint32_t lo = pack_bf16(o[0], o[1]), hi = pack_bf16(o[2], o[3]);
    if (vec >= 4) {
      *reinterpret_cast<u32x2*>(q) = u32x2{lo, hi};
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (v < left) q[v].bits = static_cast<uint16_t>((v < 2 ? lo : hi) >> (16 * (v & 1)));
    }
  }
}

// fp32 value of a scale: fp32 itself, or e8m0 (2^(b - 127), 255: NaN)
template <bool E8>
__device__ __forceinline__ float scale_at(const void* p, long long i) {
  if constexpr (E8) {
    const uint32_t b = static_cast<const uint8_t*>(p)[i];
    return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
  } else {
    return static_cast<const float*>(p)[i];
  }
}

// Stores a BM x BN tile of bf16 results through workgroup memory: written as
// the matrix instructions leave them (4 columns of 16 rows per instruction) a
// wave would touch 32 bytes of a row at a time, which HBM takes at a quarter
// of its rate. NT threads; put(row, column, 4 values) fills the tile, then
// whole rows go out 16 bytes per lane. So that 16 rows written at one column
// touch different banks, chunk c of row m lies at c ^ (m & 15) where a row is
// a power of two of chunks, and rows are one chunk longer where it is not.
template <int BM, int BN, int NT>
struct TileStore {
  static constexpr int CH = BN / 8;  // 16-byte chunks per row
  static constexpr bool POW2 = (CH & (CH - 1)) == 0;
  static constexpr int MASK = POW2 ? (CH < 16 ? CH : 16) - 1 : 0, ROW = POW2 ? CH : CH + 1;
  static constexpr int CHUNKS = BM * ROW;
  i32x4* lds;
  __device__ __forceinline__ void put(int m, int n, const float (&o)[4]) {
    const int c = n >> 3;
    reinterpret_cast<u32x2*>(lds + m * ROW + (c ^ (m & MASK)))[(n >> 2) & 1] =
        u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
  }
  // stream: y is larger than the last-level cache and so is not kept in L2,
  // where it would displace the operands (2 % of the time of a 1 GB result)
  __device__ __forceinline__ void flush(void* y, long long m0, int n0, int mrows, int ncols, int N, int stream, int tid) {
    // rows past the tile's last are past the extent, columns past N are not sent
    const __amdgpu_buffer_rsrc_t to =
        make_rsrc(static_cast<uint16_t*>(y) + m0 * N + n0, static_cast<uint32_t>((min(mrows, BM) - 1) * N + min(ncols, BN)) * 2);
    static_assert(BM * CH % NT == 0, "whole rounds");
#pragma unroll
    for (int i = 0; i < BM * CH / NT; ++i) {
      const int e = tid + NT * i, m = e / CH, c = e % CH;
      if (c * 8 < ncols) {
        const i32x4 v = lds[m * ROW + (c ^ (m & MASK))];
        const uint32_t at = static_cast<uint32_t>(m * N + c * 8) * 2;
        if (stream) __builtin_amdgcn_raw_buffer_store_b128(v, to, at, 0, kBufNT);
        else __builtin_amdgcn_raw_buffer_store_b128(v, to, at, 0, 0);
      }
    }
  }
};

// 32 e4m3 values widened to bf16, which holds each of them
__device__ __forceinline__ void widen(const i32x8& v, bf16x8 (&o)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t q = static_cast<uint32_t>(v[2 * j + i]);
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, 1.0f, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, 1.0f, true);
      o[j][4 * i] = lo.x;
      o[j][4 * i + 1] = lo.y;
      o[j][4 * i + 2] = hi.x;
      o[j][4 * i + 3] = hi.y;
    }
}

// How a 16 x 16 tile takes its 128-block: the 8-bit instruction and an fp32
// multiply-add with the scales, the 8-bit instruction with e8m0 scales of its
// own, or exact products (bf16) and the multiply-add
enum { kMulScale = 0, kMulE8m0 = 1, kMulExact = 2 };

// fragments of one operand: 32 bytes per lane of row lane % 16
template <int MODE>
struct Frag {
  i32x8 v;
  __device__ __forceinline__ void set(const i32x4& lo, const i32x4& hi) {
    v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};
template <>
struct Frag<kMulExact> {
  bf16x8 v[4];
  __device__ __forceinline__ void set(const i32x4& lo, const i32x4& hi) {
    widen(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), v);
  }
};
template <int MODE>
__device__ __forceinline__ f32x4 tile_product(const Frag<MODE>& w, const Frag<MODE>& a) {
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (MODE == kMulExact) {
#pragma unroll
    for (int j = 0; j < 4; ++j) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[j], a.v[j], d, 0, 0, 0);
  } else {
    d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, a.v, d, 0, 0, 0, 0, 0, 0);
  }
  return d;
}

// 16 bytes of a row from column k on, zeros past column K, at any alignment
__device__ __forceinline__ i32x4 load16(const uint8_t* row, int k, int K) {
  i32x4 v = {0, 0, 0, 0};
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else if (k < K) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k + i < K) v[i / 4] |= static_cast<int>(static_cast<uint32_t>(row[k + i]) << (8 * (i % 4)));
  }
  return v;
}

// Tiles in the order of their numbers run near each other in time. Workgroup
// i runs on XCD i % 8, each with an L2 of its own: consecutive numbers go to
// one XCD, and 8 row tiles by as many column tiles as it takes follow each
// other, so that an XCD's workgroups share the panels in its L2.
__device__ __forceinline__ void tile_of(unsigned int id, unsigned int ntm, unsigned int ntn, int* tm, int* tn) {
  const unsigned int total = ntm * ntn, per = total / 8, rest = total % 8, x = id % 8, l = id / 8;
  const unsigned int t = x * per + min(x, rest) + l;
  const unsigned int grp = t / (8 * ntn), m0 = grp * 8, gm = min(ntm - m0, 8u), u = t - grp * 8 * ntn;
  *tm = static_cast<int>(m0 + u % gm);
  *tn = static_cast<int>(u / gm);
}

// The shape of a tile: waves along n and m, 16 x 16 tiles per wave along n and
// m; KS groups of such waves, each with every KS-th block of K
template <int WN_, int WM_, int TN_, int TM_, int KS_>
struct MatmulShape {
  static constexpr int WN = WN_, WM = WM_, TN = TN_, TM = TM_, KS = KS_;
  static constexpr int BN = WN * TN * 16, BM = WM * TM * 16, NT = 64 * WN * WM;  // NT: threads of a group
};

// Products between the few rows and the large tiles, unaligned operands and
// fp32 results: BM x BN of y per workgroup, bound by the latency of a step's
// loads (256 x 4096 x 4096: 12.4 us; 777 x 1000 x 1333 to fp32: 14.6 us). Each
// step brings 128 columns of both operands into workgroup memory while the
// matrix cores work on the step before (two buffers); DIRECT: by 16-byte loads
// that write there without passing through registers, where every row is
// aligned for them, else through registers. 16-byte chunk c of row q lies at
// position c ^ (q & 7) of its 128 bytes, so that 8 rows read at one c touch
// different banks.
// ROWS: rows of w that share a scale, 128 (uniform per wave: TN * 16 <= 64
// columns that start at a multiple of that) or 1.
template <class S, int MODE, bool E8, int ROWS, bool F32OUT, bool DIRECT>
struct Matmul {
  static constexpr int BN = S::BN, BM = S::BM, NT = S::NT, TN = S::TN, TM = S::TM, KS = S::KS;
  static constexpr int LN = BN * 8 / NT, LM = BM * 8 / NT;  // 16-byte chunks per thread
  static_assert(TN * 16 <= 64, "one scale block of w per wave");
  static_assert(NT % 64 == 0, "a thread's rows share their low 3 bits");
  typedef std::conditional_t<MODE == kMulE8m0, int, float> SV;
  // e8m0 rows of w scale the first operand's rows, lane % 16; fp32 ones the
  // result's rows, 4 per lane
  static constexpr int NSW = ROWS == 128 ? 1 : MODE == kMulE8m0 ? TN : TN * 4;
  typedef __attribute__((address_space(3))) void lds_void;

  MatmulArgs p;
  int tid, wave, r, g, m0, n0, wn, wm, mrows, nrows;
  __amdgpu_buffer_rsrc_t rsa, rsw;
  uint32_t v0;  // the thread's first chunk
  int q0, c0;
  i32x4 ra[DIRECT ? 1 : LM], rw[DIRECT ? 1 : LN];  // in flight
  SV fsa[TM], fsw[NSW];                            // scales in flight
  f32x4 acc[TN][TM];

  // thread's chunk i: row (tid + NT i) / 8, position tid % 8, column chunk c0
  __device__ __forceinline__ void fetch(int kb, i32x4* sw, i32x4* sa) {
    if constexpr (DIRECT) {
      // the row is in the lane's offset, which the extent is checked against;
      // the column's block, the uniform offset, is not. Extents stay below 2^31.
      const bool in = kb * 128 + c0 * 16 < p.K;
      const int so = kb < p.KB ? kb * 128 : 0;
#pragma unroll
      for (int i = 0; i < LN; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsw, (lds_void*)(sw + wave * 64 + NT * i), 16,
                                                 in ? v0 + static_cast<uint32_t>(i * (NT / 8)) * p.K : 0x80000000u,
                                                 so, 0, 0);
#pragma unroll
      for (int i = 0; i < LM; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (lds_void*)(sa + wave * 64 + NT * i), 16,
                                                 in ? v0 + static_cast<uint32_t>(i * (NT / 8)) * p.K : 0x80000000u,
                                                 so, 0, 0);
    } else {
      const uint8_t* abase = p.a + static_cast<long long>(m0) * p.K;
      const uint8_t* wbase = p.w + static_cast<long long>(n0) * p.K;
#pragma unroll
      for (int i = 0; i < LN; ++i) {
        const int q = q0 + i * (NT / 8);
        rw[i] = load16(wbase + static_cast<long long>(min(q, nrows - 1)) * p.K, kb * 128 + c0 * 16, p.K);
      }
#pragma unroll
      for (int i = 0; i < LM; ++i) {
        const int q = q0 + i * (NT / 8);
        ra[i] = load16(abase + static_cast<long long>(min(q, mrows - 1)) * p.K, kb * 128 + c0 * 16, p.K);
      }
    }
  }
  __device__ __forceinline__ void land(i32x4* sw, i32x4* sa) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int i = 0; i < LN; ++i) sw[tid + NT * i] = rw[i];
#pragma unroll
      for (int i = 0; i < LM; ++i) sa[tid + NT * i] = ra[i];
    }
  }
  __device__ __forceinline__ SV scale_of(const void* q, long long i) const {
    if constexpr (MODE == kMulE8m0) return static_cast<const uint8_t*>(q)[i];
    else return scale_at<E8>(q, i);
  }
  __device__ __forceinline__ void scales(int k) {
    const int kb = min(k, p.KB - 1);
#pragma unroll
    for (int j = 0; j < TM; ++j)
      fsa[j] = scale_of(p.sa, static_cast<long long>(kb) * p.M + min(m0 + wm + 16 * j + r, p.M - 1));
    if constexpr (ROWS == 128) {
      fsw[0] = scale_of(p.sw, static_cast<long long>(min(n0 + wn, p.N - 1) / 128) * p.KB + kb);
    } else {
#pragma unroll
      for (int i = 0; i < NSW; ++i) {
        const int n = MODE == kMulE8m0 ? 16 * i + r : 16 * (i / 4) + 4 * g + i % 4;
        fsw[i] = scale_of(p.sw, static_cast<long long>(min(n0 + wn + n, p.N - 1)) * p.KB + kb);
      }
    }
  }
  // One step: the next block's loads into nw and na, this block's products
  // from cw and ca. The pointers' restrict is what lets the compiler read this
  // block while the next one's loads write workgroup memory.
  __device__ __forceinline__ void step(int kb, const i32x4* __restrict__ cw, const i32x4* __restrict__ ca,
                                       i32x4* __restrict__ nw, i32x4* __restrict__ na) {
    SV csa[TM], csw[NSW];
#pragma unroll
    for (int j = 0; j < TM; ++j) csa[j] = fsa[j];
#pragma unroll
    for (int i = 0; i < NSW; ++i) csw[i] = fsw[i];
    if (kb + KS < p.KB + KS - 1) {  // another group may have a block where this one has none
      fetch(kb + KS, nw, na);
      scales(kb + KS);
    }
    // lane's two chunks of a row of its tile 0; tile i: 128 i further
    const int bw0 = (wn + r) * 8 + (g ^ (r & 7)), bw1 = (wn + r) * 8 + ((g + 4) ^ (r & 7));
    const int ba0 = (wm + r) * 8 + (g ^ (r & 7)), ba1 = (wm + r) * 8 + ((g + 4) ^ (r & 7));
    if (kb < p.KB) {
    Frag<MODE> fw[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i) fw[i].set(cw[bw0 + 128 * i], cw[bw1 + 128 * i]);
    i32x4 lo = ca[ba0], hi = ca[ba1];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      Frag<MODE> fa;
      fa.set(lo, hi);
      if (j + 1 < TM) {
        lo = ca[ba0 + 128 * (j + 1)];
        hi = ca[ba1 + 128 * (j + 1)];
      }
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        if constexpr (MODE == kMulE8m0) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[i].v, fa.v, acc[i][j], 0, 0, 0,
                                                                       csw[ROWS == 128 ? 0 : i], 0, csa[j]);
        } else {
          const f32x4 d = tile_product<MODE>(fw[i], fa);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[i][j][v] = fmaf(d[v], csa[j] * csw[ROWS == 128 ? 0 : 4 * i + v], acc[i][j][v]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    }
    if (kb + KS < p.KB + KS - 1) land(nw, na);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): the loads into workgroup memory are done
    __syncthreads();
  }

  __device__ __forceinline__ void run(i32x4* lds) {
    constexpr int HALF = (BN + BM) * 8;
    const int kg = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / NT);  // the wave's group
    i32x4* const all = lds;
    lds += kg * 2 * HALF;
    tid = static_cast<int>(threadIdx.x) - kg * NT;
    const int lane = tid & 63;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    r = lane & 15;
    g = lane >> 4;
    int tm, tn;
    tile_of(blockIdx.x, (p.M + BM - 1) / BM, (p.N + BN - 1) / BN, &tm, &tn);
    m0 = tm * BM;
    n0 = tn * BN;
    wn = (wave % S::WN) * TN * 16;
    wm = (wave / S::WN) * TM * 16;
    mrows = min(p.M - m0, BM);
    nrows = min(p.N - n0, BN);
    q0 = tid >> 3;
    c0 = (tid & 7) ^ (q0 & 7);
    v0 = static_cast<uint32_t>(q0) * p.K + c0 * 16;
    rsa = make_rsrc(p.a + static_cast<long long>(m0) * p.K, static_cast<uint32_t>(mrows) * p.K);
    rsw = make_rsrc(p.w + static_cast<long long>(n0) * p.K, static_cast<uint32_t>(nrows) * p.K);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    fetch(kg, lds, lds + BN * 8);
    scales(kg);
    land(lds, lds + BN * 8);
    __builtin_amdgcn_s_waitcnt(0x0f70);
    __syncthreads();
    int odd = 0;  // every group takes as many steps as the first
    for (int kb = 0; kb < p.KB; kb += KS, odd ^= 1) {
      i32x4* c = lds + odd * HALF;
      i32x4* n = lds + (1 - odd) * HALF;
      step(kb + kg, c, c + BN * 8, n, n + BN * 8);
    }
    if constexpr (KS > 1) {  // the groups' sums, joined in order
      f32x4* sum = reinterpret_cast<f32x4*>(all);
      constexpr int PER = TN * TM * NT;
      static_assert((KS - 1) * PER <= KS * 2 * HALF, "the sums fit where the blocks were");
      if (kg > 0) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int j = 0; j < TM; ++j) sum[(kg - 1) * PER + (i * TM + j) * NT + tid] = acc[i][j];
      }
      __syncthreads();
      if (kg == 0) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int k = 0; k < KS - 1; ++k) acc[i][j] += sum[k * PER + (i * TM + j) * NT + tid];
      }
      __syncthreads();
    }
    const bool whole = !F32OUT && p.vec == 8;  // the last step ended with a barrier
    TileStore<BM, BN, NT> st{all};
    if (kg > 0) {
      if (whole) __syncthreads();
      return;
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int n = n0 + wn + 16 * i + 4 * g;
      float bv[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) bv[v] = p.bias && n + v < p.N ? p.bias[n + v] : 0.0f;
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const long long m = m0 + wm + 16 * j + r;
        float o[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = acc[i][j][v] + bv[v];
        if (whole) st.put(wm + 16 * j + r, n - n0, o);
        else if (m < p.M && n < p.N) store_row4<F32OUT>(p.y, m * p.N + n, p.N - n, p.vec, o);
      }
    }
    if (whole) {
      __syncthreads();
      st.flush(p.y, m0, n0, mrows, p.N - n0, p.N, p.stream, tid);
    }
  }
};

template <class S, int MODE, bool E8, int ROWS, bool F32OUT, bool DIRECT>
__global__ void __launch_bounds__(S::NT * S::KS) matmul_kernel(const MatmulArgs p) {
  __shared__ i32x4 lds[S::KS * 2 * (S::BN + S::BM) * 8];
  Matmul<S, MODE, E8, ROWS, F32OUT, DIRECT> m;
  m.p = p;
  m.run(lds);
}

// ---------------------------------------------------------------------------
// Large products: 256 rows by 64 TN columns of y by 8 waves (4 along n, 2
// along m; 16 TN x 128 each), two waves per SIMD. What bounds it is the time
// from the issue of a block's loads to their arrival, about a step and a half
// of products, and workgroup memory holds two blocks only. So a step has two halves: the first
// multiplies the wave's w rows by the first half of its a rows, the second by
// the other half. After the first half nobody needs this block's w and first
// a rows any more (w's stay in registers), and their place takes the block
// after the next; the place of the second a rows is taken one half later.
// Every load so has a step and a half to arrive, and the waits count the loads
// that may still be on their way. 32768 x 16384 x 4096 with e8m0 scales takes
// 1.84 to 1.92 ms (2290 to 2390 TFLOP/s, by the box), 4096 x 6144 x 2048 with
// fp32 scales 61 to 66 us (1570 to 1690);
// with 32 or 16 blocks of K, what a tile costs before its first product and
// behind its last (5 us) is a sixth to a third of its time.
template <int TN, int MODE, bool E8, int ROWS>
struct MatmulLarge {
  static constexpr int BN = 64 * TN, BM = 256, NT = 512, TM = 8, WC = 16 * TN;
  // 16-byte chunks of one buffer: w, then the first and the second a rows of both waves along m
  static constexpr int OX0 = BN * 8, OX1 = OX0 + BM * 4, BUF = OX1 + BM * 4;
  static constexpr int SB = MODE == kMulE8m0 ? 1 : 4;      // bytes of a scale in workgroup memory
  static constexpr int SCH = 256 * SB;  // bytes of 256 scales: two buffers for a, two for w
  static constexpr int NWL = TN, NXL = 2;  // loads per thread: w, half of a
  // loads that may be on their way when a half step begins: this or the next
  // block's second a rows, and w and the first a rows of the next block
  static constexpr int WAIT = 0x0f70 | (NWL + 2 * NXL);
  // a lane's scales of w: with one per block, 64 columns are in one block, 48 may be in two
  static constexpr int NB = TN == 4 ? 1 : TN, NSC = ROWS == 128 ? NB : SB == 1 ? 1 : 4 * TN;
  static constexpr int TILE_BUF = TileStore<BM, BN, NT>::CHUNKS, LDS = 2 * BUF > TILE_BUF ? 2 * BUF : TILE_BUF;
  typedef __attribute__((address_space(3))) void lds_void;

  MatmulArgs p;
  int tid, wave, r, g, m0, n0, wni, wmi;
  __amdgpu_buffer_rsrc_t rsa, rsw;
  uint32_t v0;
  int c16;                 // the thread's column within a block, bytes
  f32x4 acc[TN][TM];
  i32x8 fw[TN];
  uint32_t vs;  // scale on its way: of row tid (first half of the threads), of a column or block of w (second)
  f32x4 d[MODE == kMulE8m0 ? 1 : TN];  // products not yet scaled: of row tile dj, by ds

  __device__ __forceinline__ void load_w(int kb, i32x4* buf) {
    const bool in = kb * 128 + c16 < p.K;
    const int so = kb < p.KB ? kb * 128 : 0;
#pragma unroll
    for (int i = 0; i < NWL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsw, (lds_void*)(buf + wave * 64 + NT * i), 16,
                                               in ? v0 + static_cast<uint32_t>(i * 64) * p.K : 0x80000000u, so, 0, 0);
  }
  // rows 64 half + (0..63) of both 128-row parts
  __device__ __forceinline__ void load_a(int kb, int half, i32x4* buf) {
    const bool in = kb * 128 + c16 < p.K;
    const int so = kb < p.KB ? kb * 128 : 0;
#pragma unroll
    for (int i = 0; i < NXL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (lds_void*)(buf + (half ? OX1 : OX0) + wave * 64 + NT * i), 16,
                                               in ? v0 + static_cast<uint32_t>(i * 128 + half * 64) * p.K : 0x80000000u,
                                               so, 0, 0);
  }
  static __device__ __forceinline__ uint32_t raw_scale(const void* q, long long i) {
    if constexpr (MODE == kMulE8m0) return static_cast<const uint8_t*>(q)[i];
    else return __float_as_uint(scale_at<E8>(q, i));
  }
  __device__ __forceinline__ void load_scales(int kb) {
    const int k = min(kb, p.KB - 1), t = tid & 255;
    const void* q = p.sa;
    long long at = static_cast<long long>(k) * p.M + min(m0 + t, p.M - 1);
    if (tid >= 256) {
      q = p.sw;
      at = ROWS == 1 ? min(n0 + t, p.N - 1) : min(n0 + (t & 15) * 16, p.N - 1) / 128;
      at = at * p.KB + k;
    }
    vs = raw_scale(q, at);
  }
  // row 16 j + r of a wave's rows lies at 8 r + j, so that a lane's 8 scales
  // are consecutive; e8m0 column 16 i + r of a wave's columns at 4 r + i, fp32
  // columns in order; with one scale per block, those of 16 columns each
  __device__ __forceinline__ void land_scales(int kb, char* scales) {
    const int t = tid & 255;
    const int pa = (t & 128) + (t & 15) * 8 + ((t >> 4) & 7);
    const int pw = ROWS == 128 ? t & 15 : MODE == kMulE8m0 ? t / WC * 64 + (t & 15) * 4 + t % WC / 16 : t;
    char* to = scales + ((tid < 256 ? 0 : 2) + (kb & 1)) * SCH;
    const int at = tid < 256 ? pa : pw;
    if (tid >= 256 && t >= BN) return;
    if constexpr (SB == 1) reinterpret_cast<uint8_t*>(to)[at] = static_cast<uint8_t>(vs);
    else reinterpret_cast<uint32_t*>(to)[at] = vs;
  }

  // acc of row tile j += d * its scale * the columns' scales
  __device__ __forceinline__ void scale_add(int j, float sj, const uint32_t (&csw)[NSC]) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        acc[i][j][v] = fmaf(d[i][v], sj * __uint_as_float(csw[ROWS == 128 ? i % NB : 4 * i + v]), acc[i][j][v]);
  }
  // the products up to here are issued before what follows: keeps the
  // compiler from moving them behind the next barrier
  __device__ __forceinline__ void pin(int j) {
#pragma unroll
    for (int i = 0; i < TN; ++i) __asm__ volatile("" : "+v"(acc[i][j]));
  }
  // 4 row tiles of the wave by its 4 column tiles. With fp32 scales the
  // products of a row tile are scaled and added under those of the next.
  template <int HALF>
  __device__ __forceinline__ void products(const i32x4* __restrict__ x, const i32x4 (&sc)[SB == 1 ? 1 : 2],
                                           const uint32_t (&csw)[NSC]) {
    const int b0 = (wmi * 64 + r) * 8 + (g ^ (r & 7)), b1 = (wmi * 64 + r) * 8 + ((g + 4) ^ (r & 7));
    i32x4 lo = x[b0], hi = x[b1];
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const int j = HALF * 4 + jj;
      const i32x8 fa = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      if (jj < 3) {
        lo = x[b0 + 128 * (jj + 1)];
        hi = x[b1 + 128 * (jj + 1)];
      }
      if constexpr (MODE == kMulE8m0) {
        const int sj = sc[0][HALF];
#pragma unroll
        for (int i = 0; i < TN; ++i) mfma_e8(acc[i][j], fw[i], fa, static_cast<int>(csw[ROWS == 128 ? i % NB : 0]), i, sj, jj);
        pin(j);
      } else {
        f32x4 dn[TN];
#pragma unroll
        for (int i = 0; i < TN; ++i) {
          const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
          dn[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[i], fa, z, 0, 0, 0, 0, 0, 0);
        }
        if (j > 0) {
          scale_add(j - 1, __int_as_float(sc[(j - 1) / 4][(j - 1) % 4]), csw);
          pin(j - 1);
        }
#pragma unroll
        for (int i = 0; i < TN; ++i) d[i] = dn[i];
        if (j == TM - 1) scale_add(j, __int_as_float(sc[1][3]), csw);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // the instruction takes the byte of a scale register as an immediate; a
  // block's scale is in byte 0 of its register whatever the column tile
  static __device__ __forceinline__ void mfma_e8(f32x4& c, const i32x8& w, const i32x8& a, int sw, int i, int sa, int j) {
#define PARARNN_MFMA(I, J) \
  c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 0, 0, ROWS == 128 ? 0 : I, sw, J, sa)
#define PARARNN_MFMA_J(I) \
  if (j == 0) PARARNN_MFMA(I, 0); else if (j == 1) PARARNN_MFMA(I, 1); else if (j == 2) PARARNN_MFMA(I, 2); else PARARNN_MFMA(I, 3)
    if (i == 0) { PARARNN_MFMA_J(0); } else if (i == 1) { PARARNN_MFMA_J(1); } else if (i == 2) { PARARNN_MFMA_J(2); } else { PARARNN_MFMA_J(3); }
#undef PARARNN_MFMA_J
#undef PARARNN_MFMA
  }

  // Orders workgroup memory between the waves, and only that: unlike a fence
  // it leaves the loads into it that are counted separately on their way.
  static __device__ __forceinline__ void hand_over() {
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __asm__ volatile("" ::: "memory");
  }

  // One block. rd and wr are the same memory, and so are rs and ws: restrict
  // says that what is written (by the loads into workgroup memory, which the
  // compiler would otherwise wait for) does not change what is still read
  // before the next barrier. The offsets of the buffers are opaque, so that
  // nothing read in one step is taken for known in a later one.
  __device__ __forceinline__ void step(int kb, const i32x4* __restrict__ rd, i32x4* __restrict__ wr,
                                       const char* __restrict__ rs, char* __restrict__ ws) {
    int cur = (kb & 1) * BUF;
    __asm__ volatile("" : "+s"(cur));
    const int nxt = BUF - cur;
    // first half: w and the first a rows of this block have arrived, and the
    // next block's scales; 8 newer loads may not have
    __builtin_amdgcn_s_waitcnt(WAIT);
    land_scales(kb + 1, ws);
    hand_over();
    load_scales(kb + 2);
    __builtin_amdgcn_sched_barrier(0);
    load_a(kb + 1, 1, wr + nxt);
    i32x4 sc[SB == 1 ? 1 : 2];
    uint32_t csw[NSC];
    {
      const char* sa = rs + (kb & 1) * SCH;
      const char* sw = rs + (2 + (kb & 1)) * SCH;
      if constexpr (SB == 1) {
        const i32x2 t = *reinterpret_cast<const i32x2*>(sa + wmi * 128 + r * 8);
        sc[0] = i32x4{t.x, t.y, 0, 0};
      } else {
        sc[0] = *reinterpret_cast<const i32x4*>(sa + (wmi * 128 + r * 8) * 4);
        sc[1] = *reinterpret_cast<const i32x4*>(sa + (wmi * 128 + r * 8) * 4 + 16);
      }
      if constexpr (ROWS == 128) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          if constexpr (SB == 1) csw[i] = static_cast<uint8_t>(sw[wni * TN + i]);
          else csw[i] = reinterpret_cast<const uint32_t*>(sw)[wni * TN + i];
        }
      } else if constexpr (SB == 1) {
        csw[0] = *reinterpret_cast<const uint32_t*>(sw + wni * 64 + r * 4);
      } else {
#pragma unroll
        for (int i = 0; i < TN; ++i) {
          const i32x4 t = *reinterpret_cast<const i32x4*>(sw + (wni * WC + 16 * i + 4 * g) * 4);
#pragma unroll
          for (int v = 0; v < 4; ++v) csw[4 * i + v] = static_cast<uint32_t>(t[v]);
        }
      }
    }
    const int b0 = (wni * WC + r) * 8 + (g ^ (r & 7)), b1 = (wni * WC + r) * 8 + ((g + 4) ^ (r & 7));
#pragma unroll
    for (int i = 0; i < TN; ++i)
      fw[i] = __builtin_shufflevector(rd[cur + b0 + 128 * i], rd[cur + b1 + 128 * i], 0, 1, 2, 3, 4, 5, 6, 7);
    products<0>(rd + cur + OX0, sc, csw);
    // second half: the other a rows have arrived; again WAIT's newer loads may not have
    __builtin_amdgcn_s_waitcnt(WAIT);
    hand_over();
    load_w(kb + 2, wr + cur);
    load_a(kb + 2, 0, wr + cur);
    products<1>(rd + cur + OX1, sc, csw);
  }

  __device__ __forceinline__ void run(i32x4* lds, char* scales) {
    tid = threadIdx.x;
    const int lane = tid & 63;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    r = lane & 15;
    g = lane >> 4;
    wni = wave & 3;
    wmi = wave >> 2;
    int tm, tn;
    tile_of(blockIdx.x, (p.M + BM - 1) / BM, (p.N + BN - 1) / BN, &tm, &tn);
    m0 = tm * BM;
    n0 = tn * BN;
    const int q0 = tid >> 3;
    c16 = ((tid & 7) ^ (q0 & 7)) * 16;
    v0 = static_cast<uint32_t>(q0) * p.K + c16;
    rsa = make_rsrc(p.a + static_cast<long long>(m0) * p.K, static_cast<uint32_t>(min(p.M - m0, BM)) * p.K);
    rsw = make_rsrc(p.w + static_cast<long long>(n0) * p.K, static_cast<uint32_t>(min(p.N - n0, BN)) * p.K);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // in the order that the steps count them in; the bias waits in workgroup memory
    float* s_bias = reinterpret_cast<float*>(scales + 4 * SCH);
    const float bias = p.bias && tid < BN && n0 + tid < p.N ? p.bias[n0 + tid] : 0.0f;
    load_scales(0);
    const uint32_t vs0 = vs;
    load_w(0, lds);
    load_a(0, 0, lds);
    load_scales(1);
    __builtin_amdgcn_sched_barrier(0);
    load_a(0, 1, lds);
    load_w(1, lds + BUF);
    load_a(1, 0, lds + BUF);
    const uint32_t vs1 = vs;
    vs = vs0;
    land_scales(0, scales);
    vs = vs1;
    if (tid < BN) s_bias[tid] = bias;
    for (int kb = 0; kb < p.KB; ++kb) step(kb, lds, lds, scales, scales);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // no load into workgroup memory outlives the products
    const bool whole = p.vec == 8;
    TileStore<BM, BN, NT> st{lds};
    if (whole) __syncthreads();
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int n = n0 + wni * WC + 16 * i + 4 * g;
      const f32x4 bv = *reinterpret_cast<const f32x4*>(s_bias + (n - n0));
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const long long m = m0 + wmi * 128 + 16 * j + r;
        float o[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = acc[i][j][v] + bv[v];
        if (whole) st.put(wmi * 128 + 16 * j + r, n - n0, o);
        else if (m < p.M && n < p.N) store_row4<false>(p.y, m * p.N + n, p.N - n, p.vec, o);
      }
    }
    if (whole) {
      __syncthreads();
      st.flush(p.y, m0, n0, p.M - m0, p.N - n0, p.N, p.stream, tid);
    }
  }
};

template <int TN, int MODE, bool E8, int ROWS>
__global__ void __launch_bounds__(512) matmul_large_kernel(const MatmulArgs p) {
  typedef MatmulLarge<TN, MODE, E8, ROWS> M;
  // one array: what the compiler derives from several would replace what restrict says
  __shared__ i32x4 lds[M::LDS + 4 * M::SCH / 16 + 64];
  M m;
  m.p = p;
  m.run(lds, reinterpret_cast<char*>(lds + M::LDS));
}

// ---------------------------------------------------------------------------
// Few rows (up to 16 MT): the product is the time it takes to read w. A
// workgroup of 8 waves takes 16 NT columns of y; its waves take the 128-blocks
// of K in turn, straight from HBM into registers (nothing of w is used twice),
// and their sums are joined in order through workgroup memory. UN blocks are
// in flight per wave. 16 x 16384 x 4096 takes 12.6 us (5.4 TB/s of w and y).
template <int MODE, bool E8, int ROWS, bool F32OUT, int MT, int NT, int UN>
__global__ void __launch_bounds__(512) matmul_few_kernel(const MatmulArgs p) {
  constexpr int W = 8;
  __shared__ f32x4 s_acc[W][NT * MT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = static_cast<int>(blockIdx.x) * 16 * NT;
  f32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // rows past the end read the last row, and are not stored
  const uint8_t* wp[NT];
  const uint8_t* ap[MT];
#pragma unroll
  for (int i = 0; i < NT; ++i) wp[i] = p.w + static_cast<long long>(min(n0 + 16 * i + r, p.N - 1)) * p.K;
#pragma unroll
  for (int j = 0; j < MT; ++j) ap[j] = p.a + static_cast<long long>(min(16 * j + r, p.M - 1)) * p.K;

  // the two 16-byte chunks g and g + 4 of a row's block; past column K zeros (K is a multiple of 16)
  auto ld = [&](const uint8_t* row, int kb, i32x4& lo, i32x4& hi) {
    const int k0 = kb * 128 + 16 * g, k1 = k0 + 64;
    const i32x4 z = {0, 0, 0, 0};
    lo = k0 < p.K ? *reinterpret_cast<const i32x4*>(row + k0) : z;
    hi = k1 < p.K ? *reinterpret_cast<const i32x4*>(row + k1) : z;
  };
  for (int kb0 = wave * UN; kb0 < p.KB; kb0 += W * UN) {
    i32x4 wl[UN][NT], wh[UN][NT], al[UN][MT], ah[UN][MT];
    float sa[UN][MT], sw[UN][ROWS == 128 ? 1 : NT * 4];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int kb = kb0 + u;
#pragma unroll
      for (int i = 0; i < NT; ++i) ld(wp[i], kb, wl[u][i], wh[u][i]);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int kb = kb0 + u, k = min(kb, p.KB - 1);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        ld(ap[j], kb, al[u][j], ah[u][j]);
        sa[u][j] = scale_at<E8>(p.sa, static_cast<long long>(k) * p.M + min(16 * j + r, p.M - 1));
      }
      if constexpr (ROWS == 128) {
        sw[u][0] = scale_at<E8>(p.sw, static_cast<long long>(min(n0, p.N - 1) / 128) * p.KB + k);
      } else {
#pragma unroll
        for (int i = 0; i < NT * 4; ++i)
          sw[u][i] = scale_at<E8>(p.sw, static_cast<long long>(min(n0 + 16 * (i / 4) + 4 * g + i % 4, p.N - 1)) * p.KB + k);
      }
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      Frag<MODE> fa[MT];
#pragma unroll
      for (int j = 0; j < MT; ++j) fa[j].set(al[u][j], ah[u][j]);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        Frag<MODE> fw;
        fw.set(wl[u][i], wh[u][i]);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const f32x4 d = tile_product<MODE>(fw, fa[j]);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            // a block past the end adds nothing, whatever its (clamped) scale is
            const float s = sa[u][j] * sw[u][ROWS == 128 ? 0 : 4 * i + v];
            acc[i][j][v] = kb0 + u < p.KB ? fmaf(d[v], s, acc[i][j][v]) : acc[i][j][v];
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) s_acc[wave][i * MT + j][lane] = acc[i][j];
  __syncthreads();
  // wave w joins tiles w, w + 8, ...
#pragma unroll
  for (int t0 = 0; t0 < NT * MT; t0 += W) {
    const int t = t0 + wave;
    if (t >= NT * MT) break;
    const int i = t / MT, j = t % MT;
    const int n = n0 + 16 * i + 4 * g, m = 16 * j + r;
    f32x4 v = s_acc[0][t][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += s_acc[w][t][lane];
    if (m < p.M && n < p.N) {
      float o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = v[q] + (p.bias && n + q < p.N ? p.bias[n + q] : 0.0f);
      store_row4<F32OUT>(p.y, static_cast<long long>(m) * p.N + n, p.N - n, p.vec, o);
    }
  }
}

}  // namespace pararnn
