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

#include "matmul_tiles.h"

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

// Products between the few rows and the large tiles, unaligned operands and
// fp32 results: BM x BN of y per workgroup, bound by the latency of a step's
// loads (256 x 4096 x 4096: 12.4 us; 777 x 1000 x 1333 to fp32: 14.6 us).
// ROWS: rows of w that share a scale, 128 (uniform per wave: TN * 16 <= 64
// columns that start at a multiple of that) or 1.
template <class S, int MODE, bool E8, int ROWS, bool F32OUT, bool DIRECT>
struct Matmul : SmallTiles<MatmulArgs, S, DIRECT> {
  typedef SmallTiles<MatmulArgs, S, DIRECT> T;
  using T::p, T::kg, T::r, T::g, T::m0, T::n0, T::wn, T::wm;
  static constexpr int BN = S::BN, TN = S::TN, TM = S::TM, KS = S::KS;
  static_assert(TN * 16 <= 64, "one scale block of w per wave");
  typedef std::conditional_t<MODE == kMulE8m0, int, float> SV;
  // e8m0 rows of w scale the first operand's rows, lane % 16; fp32 ones the
  // result's rows, 4 per lane
  static constexpr int NSW = ROWS == 128 ? 1 : MODE == kMulE8m0 ? TN : TN * 4;

  SV fsa[TM], fsw[NSW];  // scales in flight
  f32x4 acc[TN][TM];

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
    if (T::more(kb)) {
      T::fetch(kb + KS, nw, na);
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
    if (T::more(kb)) T::land(nw, na);
    T::arrived();
  }

  __device__ __forceinline__ void run(i32x4* lds) {
    T::begin();
    i32x4* const all = lds;
    lds += kg * 2 * T::HALF;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    T::fetch(kg, lds, lds + BN * 8);
    scales(kg);
    T::land(lds, lds + BN * 8);
    T::arrived();
    int odd = 0;  // every group takes as many steps as the first
    for (int kb = 0; kb < p.KB; kb += KS, odd ^= 1) {
      i32x4* c = lds + odd * T::HALF;
      i32x4* n = lds + (1 - odd) * T::HALF;
      step(kb + kg, c, c + BN * 8, n, n + BN * 8);
    }
    T::join(acc, all);
    float bv[4];
    T::template out<F32OUT>(
        all,
        [&](int, int n) {
#pragma unroll
          for (int v = 0; v < 4; ++v) bv[v] = p.bias && n + v < p.N ? p.bias[n + v] : 0.0f;
        },
        [&](int i, int j, float(&o)[4]) {
#pragma unroll
          for (int v = 0; v < 4; ++v) o[v] = acc[i][j][v] + bv[v];
        });
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
// Large products: tiles of 256 rows by 64 TN columns. 32768 x 16384 x 4096 with e8m0 scales takes
// 1.84 to 1.92 ms (2290 to 2390 TFLOP/s, by the box), 4096 x 6144 x 2048 with
// fp32 scales 61 to 66 us (1570 to 1690);
// with 32 or 16 blocks of K, what a tile costs before its first product and
// behind its last (5 us) is a sixth to a third of its time.
template <int TN, int MODE, bool E8, int ROWS>
struct MatmulLarge : LargeTiles<MatmulArgs, TN> {
  typedef LargeTiles<MatmulArgs, TN> T;
  using T::p, T::tid, T::r, T::g, T::m0, T::n0, T::wni, T::wmi;
  static constexpr int BN = T::BN, TM = T::TM, WC = T::WC, OX0 = T::OX0, OX1 = T::OX1, BUF = T::BUF;
  static constexpr int SB = MODE == kMulE8m0 ? 1 : 4;      // bytes of a scale in workgroup memory
  static constexpr int SCH = 256 * SB;  // bytes of 256 scales: two buffers for a, two for w
  // a lane's scales of w: with one per block, 64 columns are in one block, 48 may be in two
  static constexpr int NB = TN == 4 ? 1 : TN, NSC = ROWS == 128 ? NB : SB == 1 ? 1 : 4 * TN;

  f32x4 acc[TN][TM];
  i32x8 fw[TN];
  uint32_t vs;  // scale on its way: of row tid (first half of the threads), of a column or block of w (second)
  f32x4 d[MODE == kMulE8m0 ? 1 : TN];  // products not yet scaled: of row tile dj, by ds

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
    // next block's scales; newer loads may not have
    T::wait();
    land_scales(kb + 1, ws);
    T::hand_over();
    load_scales(kb + 2);
    __builtin_amdgcn_sched_barrier(0);
    T::load_a(kb + 1, 1, wr + nxt);
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
    // second half: the other a rows have arrived; again newer loads may not have
    T::wait();
    T::hand_over();
    T::load_w(kb + 2, wr + cur);
    T::load_a(kb + 2, 0, wr + cur);
    products<1>(rd + cur + OX1, sc, csw);
  }

  __device__ __forceinline__ void run(i32x4* lds, char* scales) {
    T::begin();
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // in the order that the steps count them in; the bias waits in workgroup memory
    float* s_bias = reinterpret_cast<float*>(scales + 4 * SCH);
    const float bias = p.bias && tid < BN && n0 + tid < p.N ? p.bias[n0 + tid] : 0.0f;
    load_scales(0);
    const uint32_t vs0 = vs;
    T::load_w(0, lds);
    T::load_a(0, 0, lds);
    load_scales(1);
    __builtin_amdgcn_sched_barrier(0);
    T::load_a(0, 1, lds);
    T::load_w(1, lds + BUF);
    T::load_a(1, 0, lds + BUF);
    const uint32_t vs1 = vs;
    vs = vs0;
    land_scales(0, scales);
    vs = vs1;
    if (tid < BN) s_bias[tid] = bias;
    for (int kb = 0; kb < p.KB; ++kb) step(kb, lds, lds, scales, scales);
    T::wait_all();
    f32x4 bv;
    T::template out<false>(
        lds, [&](int, int nl) { bv = *reinterpret_cast<const f32x4*>(s_bias + nl); },
        [&](int i, int j, float(&o)[4]) {
#pragma unroll
          for (int v = 0; v < 4; ++v) o[v] = acc[i][j][v] + bv[v];
        });
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
  FewRows<MT, NT> x;
  x.begin(p, n0, r, g);
  for (int kb0 = wave * UN; kb0 < p.KB; kb0 += W * UN) {
    i32x4 wl[UN][NT], wh[UN][NT], al[UN][MT], ah[UN][MT];
    float sa[UN][MT], sw[UN][ROWS == 128 ? 1 : NT * 4];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int kb = kb0 + u;
#pragma unroll
      for (int i = 0; i < NT; ++i) x.load(x.wp[i], kb, wl[u][i], wh[u][i]);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int kb = kb0 + u, k = min(kb, p.KB - 1);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        x.load(x.ap[j], kb, al[u][j], ah[u][j]);
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
