// matmul_tiles.h -- what the products of 8-bit matrices y^T = w a^T share,
// whatever their numbers and scales are: the order of the tiles, both operands'
// way into workgroup memory with its waits, the sums over K's groups and the
// results' way out. Args: a [M][K], w [N][K] (bytes), y [M][N], M, N, K, KB =
// ceil(K / 128), vec, stream. gfx950 (CDNA4) only.
#pragma once

#include "layer_common.h"

namespace pararnn {

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

// Tiles of BN x BM by the waves of a shape S, a block of 128 of K at a time, in
// two buffers: each step brings 128 columns of both operands into workgroup
// memory while the matrix cores work on the step before; DIRECT: by 16-byte
// loads that write there without passing through registers, where every row is
// aligned for them, else through registers. 16-byte chunk c of row q lies at
// position c ^ (q & 7) of its 128 bytes, so that 8 rows read at one c touch
// different banks.
template <class Args, class S, bool DIRECT>
struct SmallTiles {
  static constexpr int BN = S::BN, BM = S::BM, NT = S::NT, TN = S::TN, TM = S::TM, KS = S::KS;
  static constexpr int LN = BN * 8 / NT, LM = BM * 8 / NT, HALF = (BN + BM) * 8;  // 16-byte chunks: per thread, of a buffer
  static_assert(NT % 64 == 0, "a thread's rows share their low 3 bits");
  typedef __attribute__((address_space(3))) void lds_void;

  Args p;
  int kg;  // the wave's group
  int tid, wave, r, g, m0, n0, wn, wm, mrows, nrows;
  __amdgpu_buffer_rsrc_t rsa, rsw;
  uint32_t v0;  // the thread's first chunk
  int q0, c0;
  i32x4 ra[DIRECT ? 1 : LM], rw[DIRECT ? 1 : LN];  // in flight

  __device__ __forceinline__ void begin() {
    kg = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / NT);
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
  }
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
  // what came through registers
  __device__ __forceinline__ void land(i32x4* sw, i32x4* sa) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int i = 0; i < LN; ++i) sw[tid + NT * i] = rw[i];
#pragma unroll
      for (int i = 0; i < LM; ++i) sa[tid + NT * i] = ra[i];
    }
  }
  // the end of a step: the loads into workgroup memory are done, for every wave
  static __device__ __forceinline__ void arrived() {
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __syncthreads();
  }
  // another group may have a block where this one has none
  __device__ __forceinline__ bool more(int kb) const { return kb + KS < p.KB + KS - 1; }
  // The groups' sums, joined in order by the first, where the blocks were; all: the workgroup's memory
  template <class V>
  __device__ __forceinline__ void join(V (&acc)[TN][TM], i32x4* all) const {
    if constexpr (KS > 1) {
      V* sum = reinterpret_cast<V*>(all);
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
  }
  // The first group's results to y: column(i, n) before those of column tile i, which begin at column n, then
  // value(i, j, o) for 4 of them in a row of row tile j. Nobody reads the blocks any more.
  template <bool F32OUT, class Column, class Value>
  __device__ __forceinline__ void out(i32x4* all, Column column, Value value) const {
    const bool whole = !F32OUT && p.vec == 8;
    TileStore<BM, BN, NT> st{all};
    if (kg > 0) {
      if (whole) __syncthreads();
      return;
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int n = n0 + wn + 16 * i + 4 * g;
      column(i, n);
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const long long m = m0 + wm + 16 * j + r;
        float o[4];
        value(i, j, o);
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

// Large tiles: 256 rows by 64 TN columns of y by 8 waves (4 along n, 2 along m;
// 16 TN x 128 each), two waves per SIMD. What bounds them is the time
// from the issue of a block's loads to their arrival, about a step and a half
// of products, and workgroup memory holds two blocks only. So a step has two halves: the first
// multiplies the wave's w rows by the first half of its a rows, the second by
// the other half. After the first half nobody needs this block's w and first
// a rows any more (w's stay in registers), and their place takes the block
// after the next; the place of the second a rows is taken one half later.
// Every load so has a step and a half to arrive, and the waits count the loads
// that may still be on their way:
//   wait(), hand_over(), load_a(kb + 1, 1, the other buffer), products of the first a rows,
//   wait(), hand_over(), load_w(kb + 2), load_a(kb + 2, 0) (this buffer), products of the second.
template <class Args, int TN>
struct LargeTiles {
  static constexpr int BN = 64 * TN, BM = 256, NT = 512, TM = 8, WC = 16 * TN;
  // 16-byte chunks of one buffer: w, then the first and the second a rows of both waves along m
  static constexpr int OX0 = BN * 8, OX1 = OX0 + BM * 4, BUF = OX1 + BM * 4;
  static constexpr int NWL = TN, NXL = 2;  // loads per thread: w, half of a
  static constexpr int TILE_BUF = TileStore<BM, BN, NT>::CHUNKS, LDS = 2 * BUF > TILE_BUF ? 2 * BUF : TILE_BUF;
  typedef __attribute__((address_space(3))) void lds_void;

  Args p;
  int tid, wave, r, g, m0, n0, wni, wmi;
  __amdgpu_buffer_rsrc_t rsa, rsw;
  uint32_t v0;
  int c16;  // the thread's column within a block, bytes

  __device__ __forceinline__ void begin() {
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
  }
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
  // Loads that may be on their way when a half step begins: this or the next
  // block's second a rows, and w and the first a rows of the next block
  static __device__ __forceinline__ void wait() { __builtin_amdgcn_s_waitcnt(0x0f70 | (NWL + 2 * NXL)); }
  // no load into workgroup memory outlives the products
  static __device__ __forceinline__ void wait_all() { __builtin_amdgcn_s_waitcnt(0x0f70); }
  // Orders workgroup memory between the waves, and only that: unlike a fence
  // it leaves the loads into it that are counted separately on their way.
  static __device__ __forceinline__ void hand_over() {
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __asm__ volatile("" ::: "memory");
  }
  // Results to y: column(i, nl) before those of column tile i, which begin at column nl of the tile, then
  // value(i, j, o) for 4 of them in a row of row tile j
  template <bool F32OUT, class Column, class Value>
  __device__ __forceinline__ void out(i32x4* lds, Column column, Value value) const {
    const bool whole = !F32OUT && p.vec == 8;
    TileStore<BM, BN, NT> st{lds};
    if (whole) __syncthreads();
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int nl = wni * WC + 16 * i + 4 * g, n = n0 + nl;
      column(i, nl);
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const long long m = m0 + wmi * 128 + 16 * j + r;
        float o[4];
        value(i, j, o);
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

// Up to 16 MT rows of a and 16 NT of w, straight from memory into registers: nothing of w is used twice
template <int MT, int NT>
struct FewRows {
  const uint8_t* wp[NT];
  const uint8_t* ap[MT];
  int K, g;
  // rows past the end read the last row, and are not stored
  template <class Args>
  __device__ __forceinline__ void begin(const Args& p, int n0, int r, int g_) {
    K = p.K;
    g = g_;
#pragma unroll
    for (int i = 0; i < NT; ++i) wp[i] = p.w + static_cast<long long>(min(n0 + 16 * i + r, p.N - 1)) * p.K;
#pragma unroll
    for (int j = 0; j < MT; ++j) ap[j] = p.a + static_cast<long long>(min(16 * j + r, p.M - 1)) * p.K;
  }
  // the two 16-byte chunks g and g + 4 of a row's block; past column K zeros (K is a multiple of 16)
  __device__ __forceinline__ void load(const uint8_t* row, int kb, i32x4& lo, i32x4& hi) const {
    const int k0 = kb * 128 + 16 * g, k1 = k0 + 64;
    const i32x4 z = {0, 0, 0, 0};
    lo = k0 < K ? *reinterpret_cast<const i32x4*>(row + k0) : z;
    hi = k1 < K ? *reinterpret_cast<const i32x4*>(row + k1) : z;
  }
};

}  // namespace pararnn
