// matmul_int8.h -- product of two 8-bit integer matrices with a scale for each
// row of both (a token and an output channel):
//   y[m][n] = sum_k a[m][k] w[n][k] * sa[m] * sw[n] + bias[n].
// The sum over k is exact, in the 32-bit integers of the matrix instructions
// (16 x 16 x 64, two for a block of 128), so the scales wait for the end: they
// and the bias are the epilogue. Operands, tiles and the order of tiles are
// those of the 8-bit floating-point product (matmul_tiles.h): a wave holds 16 x
// 16 tiles of y^T, a lane 4 consecutive columns of one row of y.
#pragma once

#include "../layer/matmul_tiles.h"

namespace pararnn {

struct Int8Args {
  const uint8_t* a;   // [M][K]
  const float* sa;    // [M]
  const uint8_t* w;   // [N][K]
  const float* sw;    // [N]
  const float* bias;  // [N] or nullptr
  void* y;            // [M][N] bf16 or fp32
  int M, N, K, KB;
  int vec;            // columns of y that go out at a time: 8, 4 or 1
  int stream;         // y is larger than the last-level cache
};

__device__ __forceinline__ i32x4 mul_block(const i32x4& wl, const i32x4& wh, const i32x4& al, const i32x4& ah, i32x4 c) {
  c = __builtin_amdgcn_mfma_i32_16x16x64_i8(wl, al, c, 0, 0, 0);
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(wh, ah, c, 0, 0, 0);
}
__device__ __forceinline__ void scaled(const i32x4& c, float sa, const float (&sw)[4], const float (&bias)[4], float (&o)[4]) {
#pragma unroll
  for (int v = 0; v < 4; ++v) o[v] = static_cast<float>(c[v]) * sa * sw[v] + bias[v];
}

// Between the few rows and the large tiles, and unaligned operands: BN x BM of
// y per workgroup; KS groups of waves take every KS-th block of K and their sums
// are joined (integers: in any order). The latency
// of the blocks bounds them: 777 x 1000 x 1333, whose rows no wide load can take, 13 us,
// 777 x 1000 x 1344 6.0.
template <class S, bool F32OUT, bool DIRECT>
struct Int8Tiles : SmallTiles<Int8Args, S, DIRECT> {
  typedef SmallTiles<Int8Args, S, DIRECT> T;
  using T::p, T::kg, T::r, T::g, T::m0, T::wn, T::wm;
  static constexpr int BN = S::BN, TN = S::TN, TM = S::TM, KS = S::KS;
  i32x4 acc[TN][TM];

  // The pointers' restrict lets reads of this block pass the next one's loads into workgroup memory.
  __device__ __forceinline__ void step(int kb, const i32x4* __restrict__ c, i32x4* __restrict__ nx) {
    // lane's two chunks of a row of its tile 0; tile i: 128 i further
    const int bw0 = (wn + r) * 8 + (g ^ (r & 7)), bw1 = (wn + r) * 8 + ((g + 4) ^ (r & 7));
    const int ba0 = (wm + r) * 8 + (g ^ (r & 7)), ba1 = (wm + r) * 8 + ((g + 4) ^ (r & 7));
    if (T::more(kb)) T::fetch(kb + KS, nx, nx + BN * 8);
    if (kb < p.KB) {
      const i32x4* ca = c + BN * 8;
      i32x4 wl[TN], wh[TN];
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        wl[i] = c[bw0 + 128 * i];
        wh[i] = c[bw1 + 128 * i];
      }
      i32x4 lo = ca[ba0], hi = ca[ba1];
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const i32x4 l = lo, h = hi;
        if (j + 1 < TM) {
          lo = ca[ba0 + 128 * (j + 1)];
          hi = ca[ba1 + 128 * (j + 1)];
        }
#pragma unroll
        for (int i = 0; i < TN; ++i) acc[i][j] = mul_block(wl[i], wh[i], l, h, acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (T::more(kb)) T::land(nx, nx + BN * 8);
    T::arrived();
  }
  __device__ __forceinline__ void run(i32x4* lds) {
    T::begin();
    i32x4* const mine = lds + kg * 2 * T::HALF;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    T::fetch(kg, mine, mine + BN * 8);
    T::land(mine, mine + BN * 8);
    T::arrived();
    int odd = 0;  // every group takes as many steps as the first
    for (int kb = 0; kb < p.KB; kb += KS, odd ^= 1) step(kb + kg, mine + odd * T::HALF, mine + (1 - odd) * T::HALF);
    T::join(acc, lds);
    float sa[TM], sw[4], bv[4];
    T::template out<F32OUT>(
        lds,
        [&](int i, int n) {
          if (i == 0) {
#pragma unroll
            for (int j = 0; j < TM; ++j) sa[j] = p.sa[min(m0 + wm + 16 * j + r, p.M - 1)];
          }
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            sw[v] = p.sw[min(n + v, p.N - 1)];
            bv[v] = p.bias && n + v < p.N ? p.bias[n + v] : 0.0f;
          }
        },
        [&](int i, int j, float(&o)[4]) { scaled(acc[i][j], sa[j], sw, bv, o); });
  }
};
template <class S, bool F32OUT, bool DIRECT>
__global__ void __launch_bounds__(S::NT * S::KS) int8_kernel(const Int8Args p) {
  typedef Int8Tiles<S, F32OUT, DIRECT> M;
  __shared__ i32x4 lds[S::KS * 2 * M::HALF];
  M m;
  m.p = p;
  m.run(lds);
}

// Large products: tiles of 256 rows by 64 TN columns. The matrix instructions bound it: 32768 x
// 16384 x 4096 in 1.79 ms, 2460 TOP/s (2030 on a warm
// card; the same product of 8-bit floating-point numbers 2290 to 2390 TFLOP/s).
template <int TN, bool F32OUT>
struct Int8Large : LargeTiles<Int8Args, TN> {
  typedef LargeTiles<Int8Args, TN> T;
  using T::p, T::tid, T::r, T::g, T::m0, T::n0, T::wni, T::wmi;
  static constexpr int BN = T::BN, TM = T::TM, WC = T::WC, OX0 = T::OX0, OX1 = T::OX1, BUF = T::BUF;
  i32x4 acc[TN][TM], wl[TN], wh[TN];

  // 4 row tiles of the wave by its TN column tiles
  template <int HALF>
  __device__ __forceinline__ void products(const i32x4* __restrict__ x) {
    const int b0 = (wmi * 64 + r) * 8 + (g ^ (r & 7)), b1 = (wmi * 64 + r) * 8 + ((g + 4) ^ (r & 7));
    i32x4 lo = x[b0], hi = x[b1];
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const int j = HALF * 4 + jj;
      const i32x4 l = lo, h = hi;
      if (jj < 3) {
        lo = x[b0 + 128 * (jj + 1)];
        hi = x[b1 + 128 * (jj + 1)];
      }
#pragma unroll
      for (int i = 0; i < TN; ++i) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wl[i], l, acc[i][j], 0, 0, 0);
#pragma unroll
      for (int i = 0; i < TN; ++i) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wh[i], h, acc[i][j], 0, 0, 0);
      // the products up to here are issued before what follows: keeps the compiler from moving them behind
      // the next barrier
#pragma unroll
      for (int i = 0; i < TN; ++i) __asm__ volatile("" : "+v"(acc[i][j]));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // One block. rd and wr are the same memory: restrict says that what the loads write does not change what is
  // still read before the next barrier. The buffer's offset is opaque, so that nothing read in one step is
  // taken for known in a later one.
  __device__ __forceinline__ void step(int kb, const i32x4* __restrict__ rd, i32x4* __restrict__ wr) {
    int cur = (kb & 1) * BUF;
    __asm__ volatile("" : "+s"(cur));
    const int nxt = BUF - cur;
    // first half: w and the first a rows of this block have arrived; newer loads may not have
    T::wait();
    T::hand_over();
    T::load_a(kb + 1, 1, wr + nxt);
    const int b0 = (wni * WC + r) * 8 + (g ^ (r & 7)), b1 = (wni * WC + r) * 8 + ((g + 4) ^ (r & 7));
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      wl[i] = rd[cur + b0 + 128 * i];
      wh[i] = rd[cur + b1 + 128 * i];
    }
    products<0>(rd + cur + OX0);
    // second half: the other a rows have arrived
    T::wait();
    T::hand_over();
    T::load_w(kb + 2, wr + cur);
    T::load_a(kb + 2, 0, wr + cur);
    products<1>(rd + cur + OX1);
  }

  __device__ __forceinline__ void run(i32x4* lds, float* rows) {
    T::begin();
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    // the rows' factors wait in workgroup memory: sa, sw, bias; loaded ahead of what the steps count
    const float f0 = tid < 256 ? p.sa[min(m0 + tid, p.M - 1)] : p.sw[min(n0 + (tid & 255), p.N - 1)];
    const float f1 = p.bias && tid < BN && n0 + tid < p.N ? p.bias[n0 + tid] : 0.0f;
    rows[tid] = f0;
    if (tid < 256) rows[512 + tid] = f1;
    T::load_w(0, lds);
    T::load_a(0, 0, lds);
    T::load_a(0, 1, lds);
    T::load_w(1, lds + BUF);
    T::load_a(1, 0, lds + BUF);
    for (int kb = 0; kb < p.KB; ++kb) step(kb, lds, lds);
    T::wait_all();
    float sa[TM], sw[4], bv[4];
#pragma unroll
    for (int j = 0; j < TM; ++j) sa[j] = rows[wmi * 128 + 16 * j + r];
    T::template out<F32OUT>(
        lds,
        [&](int, int nl) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            sw[v] = rows[256 + nl + v];
            bv[v] = rows[512 + nl + v];
          }
        },
        [&](int i, int j, float(&o)[4]) { scaled(acc[i][j], sa[j], sw, bv, o); });
  }
};

template <int TN, bool F32OUT>
__global__ void __launch_bounds__(512) int8_large_kernel(const Int8Args p) {
  typedef Int8Large<TN, F32OUT> M;
  // one array: what the compiler derives from several would replace what restrict says
  __shared__ i32x4 lds[M::LDS + 768 / 4];
  M m;
  m.p = p;
  m.run(lds, reinterpret_cast<float*>(lds + M::LDS));
}

// Few rows (up to 16 MT): the product is the time it takes to read w. A
// workgroup of 8 waves takes 16 NT columns of y; its waves take the 128-blocks
// of K in turn, straight from HBM into registers (nothing of w is used twice),
// UN blocks in flight per wave, and their sums are joined through workgroup
// memory. 16 x 16384 x 4096: 12.7 us, 5.3 TB/s of w.
template <bool F32OUT, int MT, int NT, int UN>
__global__ void __launch_bounds__(512) int8_few_kernel(const Int8Args p) {
  constexpr int W = 8;
  __shared__ i32x4 s_acc[W][NT * MT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = static_cast<int>(blockIdx.x) * 16 * NT;
  i32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  FewRows<MT, NT> x;
  x.begin(p, n0, r, g);
  for (int kb0 = wave * UN; kb0 < p.KB; kb0 += W * UN) {
    i32x4 wl[UN][NT], wh[UN][NT], al[UN][MT], ah[UN][MT];
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i) x.load(x.wp[i], kb0 + u, wl[u][i], wh[u][i]);
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int j = 0; j < MT; ++j) x.load(x.ap[j], kb0 + u, al[u][j], ah[u][j]);
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = mul_block(wl[u][i], wh[u][i], al[u][j], ah[u][j], acc[i][j]);
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
    if (m < p.M && n < p.N) {
      i32x4 v = s_acc[0][t][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) v += s_acc[w][t][lane];
      float sw[4], bv[4], o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sw[q] = p.sw[min(n + q, p.N - 1)];
        bv[q] = p.bias && n + q < p.N ? p.bias[n + q] : 0.0f;
      }
      scaled(v, p.sa[m], sw, bv, o);
      store_row4<F32OUT>(p.y, static_cast<long long>(m) * p.N + n, p.N - n, p.vec, o);
    }
  }
}

}  // namespace pararnn
