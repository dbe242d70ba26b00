// matmul_int8.h -- product of two 8-bit integer matrices with a scale for each
// row of both (a token and an output channel):
//   y[m][n] = sum_k a[m][k] w[n][k] * sa[m] * sw[n] + bias[n].
// The sum over k is exact, in the 32-bit integers of the matrix instructions
// (16 x 16 x 64, two for a block of 128), so the scales wait for the end: they
// and the bias are the epilogue. Operands, tiles and the order of tiles are
// those of the 8-bit floating-point product: a wave holds 16 x 16 tiles of y^T,
// a lane 4 consecutive columns of one row of y.
#pragma once

#include "../layer/matmul_fp8.h"

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
// y per workgroup, two buffers, as in Matmul; KS groups of waves take every
// KS-th block of K and their sums are joined (integers: in any order). The latency
// of the blocks bounds them: 777 x 1000 x 1333, whose rows no wide load can take, 13 us,
// 777 x 1000 x 1344 6.0.
template <class S, bool F32OUT, bool DIRECT>
__global__ void __launch_bounds__(S::NT * S::KS) int8_kernel(const Int8Args p) {
  constexpr int BN = S::BN, BM = S::BM, NT = S::NT, TN = S::TN, TM = S::TM, KS = S::KS;
  constexpr int LN = BN * 8 / NT, LM = BM * 8 / NT, HALF = (BN + BM) * 8;  // 16-byte chunks
  typedef __attribute__((address_space(3))) void lds_void;
  __shared__ i32x4 lds[KS * 2 * HALF];
  const int kg = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / NT);  // the wave's group
  i32x4* const mine = lds + kg * 2 * HALF;
  const int tid = static_cast<int>(threadIdx.x) - kg * NT, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int tm, tn;
  tile_of(blockIdx.x, (p.M + BM - 1) / BM, (p.N + BN - 1) / BN, &tm, &tn);
  const int m0 = tm * BM, n0 = tn * BN, mrows = min(p.M - m0, BM), nrows = min(p.N - n0, BN);
  const int wn = (wave % S::WN) * TN * 16, wm = (wave / S::WN) * TM * 16;
  // thread's chunk i: row (tid + NT i) / 8, position tid % 8, column chunk c0
  const int q0 = tid >> 3, c0 = (tid & 7) ^ (q0 & 7);
  const uint32_t v0 = static_cast<uint32_t>(q0) * p.K + c0 * 16;
  const uint8_t* const ab = p.a + static_cast<long long>(m0) * p.K;
  const uint8_t* const wb = p.w + static_cast<long long>(n0) * p.K;
  const __amdgpu_buffer_rsrc_t rsa = make_rsrc(ab, static_cast<uint32_t>(mrows) * p.K);
  const __amdgpu_buffer_rsrc_t rsw = make_rsrc(wb, static_cast<uint32_t>(nrows) * p.K);
  i32x4 ra[DIRECT ? 1 : LM], rw[DIRECT ? 1 : LN];  // in flight
  auto fetch = [&](int kb, i32x4* sw, i32x4* sa) {
    if constexpr (DIRECT) {
      // the row is in the lane's offset, which the extent is checked against; the block of columns is not
      const bool in = kb * 128 + c0 * 16 < p.K;
      const int so = kb < p.KB ? kb * 128 : 0;
#pragma unroll
      for (int i = 0; i < LN; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsw, (lds_void*)(sw + wave * 64 + NT * i), 16,
                                                 in ? v0 + static_cast<uint32_t>(i * (NT / 8)) * p.K : 0x80000000u, so, 0, 0);
#pragma unroll
      for (int i = 0; i < LM; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (lds_void*)(sa + wave * 64 + NT * i), 16,
                                                 in ? v0 + static_cast<uint32_t>(i * (NT / 8)) * p.K : 0x80000000u, so, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < LN; ++i)
        rw[i] = load16(wb + static_cast<long long>(min(q0 + i * (NT / 8), nrows - 1)) * p.K, kb * 128 + c0 * 16, p.K);
#pragma unroll
      for (int i = 0; i < LM; ++i)
        ra[i] = load16(ab + static_cast<long long>(min(q0 + i * (NT / 8), mrows - 1)) * p.K, kb * 128 + c0 * 16, p.K);
    }
  };
  auto land = [&](i32x4* sw, i32x4* sa) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int i = 0; i < LN; ++i) sw[tid + NT * i] = rw[i];
#pragma unroll
      for (int i = 0; i < LM; ++i) sa[tid + NT * i] = ra[i];
    }
  };
  i32x4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  // lane's two chunks of a row of its tile 0; tile i: 128 i further
  const int bw0 = (wn + r) * 8 + (g ^ (r & 7)), bw1 = (wn + r) * 8 + ((g + 4) ^ (r & 7));
  const int ba0 = (wm + r) * 8 + (g ^ (r & 7)), ba1 = (wm + r) * 8 + ((g + 4) ^ (r & 7));
  // The pointers' restrict lets reads of this block pass the next one's loads into workgroup memory.
  auto step = [&](int kb, const i32x4* __restrict__ c, i32x4* __restrict__ nx) {
    const bool more = kb + KS < p.KB + KS - 1;  // another group may have a block where this one has none
    if (more) fetch(kb + KS, nx, nx + BN * 8);
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
    if (more) land(nx, nx + BN * 8);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): the loads into workgroup memory are done
    __syncthreads();
  };
  fetch(kg, mine, mine + BN * 8);
  land(mine, mine + BN * 8);
  __builtin_amdgcn_s_waitcnt(0x0f70);
  __syncthreads();
  int odd = 0;  // every group takes as many steps as the first
  for (int kb = 0; kb < p.KB; kb += KS, odd ^= 1) step(kb + kg, mine + odd * HALF, mine + (1 - odd) * HALF);
  if constexpr (KS > 1) {
    constexpr int PER = TN * TM * NT;
    static_assert((KS - 1) * PER <= KS * 2 * HALF, "the sums fit where the blocks were");
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) lds[(kg - 1) * PER + (i * TM + j) * NT + tid] = acc[i][j];
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
          for (int k = 0; k < KS - 1; ++k) acc[i][j] += lds[k * PER + (i * TM + j) * NT + tid];
    }
    __syncthreads();
  }
  const bool whole = !F32OUT && p.vec == 8;  // the last step ended with a barrier
  TileStore<BM, BN, NT> st{lds};
  if (kg > 0) {
    if (whole) __syncthreads();
    return;
  }
  float sa[TM];
#pragma unroll
  for (int j = 0; j < TM; ++j) sa[j] = p.sa[min(m0 + wm + 16 * j + r, p.M - 1)];
#pragma unroll
  for (int i = 0; i < TN; ++i) {
    const int n = n0 + wn + 16 * i + 4 * g;
    float sw[4], bv[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      sw[v] = p.sw[min(n + v, p.N - 1)];
      bv[v] = p.bias && n + v < p.N ? p.bias[n + v] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const long long m = m0 + wm + 16 * j + r;
      float o[4];
      scaled(acc[i][j], sa[j], sw, bv, o);
      if (whole) st.put(wm + 16 * j + r, n - n0, o);
      else if (m < p.M && n < p.N) store_row4<F32OUT>(p.y, m * p.N + n, p.N - n, p.vec, o);
    }
  }
  if (whole) {
    __syncthreads();
    st.flush(p.y, m0, n0, mrows, p.N - n0, p.N, p.stream, tid);
  }
}

// Large products: 256 rows by 64 TN columns of y by 8 waves (4 along n, 2 along
// m), in the half steps of MatmulLarge: after the first half of a block nobody
// needs its w and first a rows any more, and the block after the next takes
// their place, so that every load has a step and a half to arrive. The matrix
// instructions bound it: 32768 x 16384 x 4096 in 1.79 ms, 2460 TOP/s (2030 on a warm
// card; the same product of 8-bit floating-point numbers 2290 to 2390 TFLOP/s).
template <int TN, bool F32OUT>
struct Int8Large {
  static constexpr int BN = 64 * TN, BM = 256, NT = 512, TM = 8, WC = 16 * TN;
  // 16-byte chunks of one buffer: w, then the first and the second a rows of both waves along m
  static constexpr int OX0 = BN * 8, OX1 = OX0 + BM * 4, BUF = OX1 + BM * 4;
  static constexpr int NWL = TN, NXL = 2;  // loads per thread: w, half of a
  // loads that may be on their way when a half step begins
  static constexpr int WAIT = 0x0f70 | (NWL + 2 * NXL);
  static constexpr int TILE_BUF = TileStore<BM, BN, NT>::CHUNKS, LDS = 2 * BUF > TILE_BUF ? 2 * BUF : TILE_BUF;
  typedef __attribute__((address_space(3))) void lds_void;

  Int8Args p;
  int tid, wave, r, g, m0, n0, wni, wmi;
  __amdgpu_buffer_rsrc_t rsa, rsw;
  uint32_t v0;
  int c16;  // the thread's column within a block, bytes
  i32x4 acc[TN][TM], wl[TN], wh[TN];

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
  // Orders workgroup memory between the waves, and only that: unlike a fence it leaves the loads into it that
  // are counted separately on their way.
  static __device__ __forceinline__ void hand_over() {
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __asm__ volatile("" ::: "memory");
  }
  // One block. rd and wr are the same memory: restrict says that what the loads write does not change what is
  // still read before the next barrier. The buffer's offset is opaque, so that nothing read in one step is
  // taken for known in a later one.
  __device__ __forceinline__ void step(int kb, const i32x4* __restrict__ rd, i32x4* __restrict__ wr) {
    int cur = (kb & 1) * BUF;
    __asm__ volatile("" : "+s"(cur));
    const int nxt = BUF - cur;
    // first half: w and the first a rows of this block have arrived; newer loads may not have
    __builtin_amdgcn_s_waitcnt(WAIT);
    hand_over();
    load_a(kb + 1, 1, wr + nxt);
    const int b0 = (wni * WC + r) * 8 + (g ^ (r & 7)), b1 = (wni * WC + r) * 8 + ((g + 4) ^ (r & 7));
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      wl[i] = rd[cur + b0 + 128 * i];
      wh[i] = rd[cur + b1 + 128 * i];
    }
    products<0>(rd + cur + OX0);
    // second half: the other a rows have arrived
    __builtin_amdgcn_s_waitcnt(WAIT);
    hand_over();
    load_w(kb + 2, wr + cur);
    load_a(kb + 2, 0, wr + cur);
    products<1>(rd + cur + OX1);
  }

  __device__ __forceinline__ void run(i32x4* lds, float* rows) {
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
      for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    // the rows' factors wait in workgroup memory: sa, sw, bias; loaded ahead of what the steps count
    const float f0 = tid < 256 ? p.sa[min(m0 + tid, p.M - 1)] : p.sw[min(n0 + (tid & 255), p.N - 1)];
    const float f1 = p.bias && tid < BN && n0 + tid < p.N ? p.bias[n0 + tid] : 0.0f;
    rows[tid] = f0;
    if (tid < 256) rows[512 + tid] = f1;
    load_w(0, lds);
    load_a(0, 0, lds);
    load_a(0, 1, lds);
    load_w(1, lds + BUF);
    load_a(1, 0, lds + BUF);
    for (int kb = 0; kb < p.KB; ++kb) step(kb, lds, lds);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // no load into workgroup memory outlives the products
    const bool whole = !F32OUT && p.vec == 8;
    TileStore<BM, BN, NT> st{lds};
    if (whole) __syncthreads();
    float sa[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) sa[j] = rows[wmi * 128 + 16 * j + r];
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int nl = wni * WC + 16 * i + 4 * g, n = n0 + nl;
      float sw[4], bv[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        sw[v] = rows[256 + nl + v];
        bv[v] = rows[512 + nl + v];
      }
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const long long m = m0 + wmi * 128 + 16 * j + r;
        float o[4];
        scaled(acc[i][j], sa[j], sw, bv, o);
        if (whole) st.put(wmi * 128 + 16 * j + r, nl, o);
        else if (m < p.M && n < p.N) store_row4<F32OUT>(p.y, m * p.N + n, p.N - n, p.vec, o);
      }
    }
    if (whole) {
      __syncthreads();
      st.flush(p.y, m0, n0, p.M - m0, p.N - n0, p.N, p.stream, tid);
    }
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
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i) ld(wp[i], kb0 + u, wl[u][i], wh[u][i]);
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int j = 0; j < MT; ++j) ld(ap[j], kb0 + u, al[u][j], ah[u][j]);
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
