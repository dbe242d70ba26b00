// delta_common.h -- operands of the delta rule's matrix instructions. gfx950
// (CDNA4) only.
//
// Sums of the delta rule are kept to fp32 on the bf16 matrix cores: an fp32
// operand is split into three bf16 planes (8 bits each: their sum is the value
// to 2^-25 of it), and a product of two split operands keeps the six products
// of planes that are above 2^-24 of the whole. A bf16 tensor is one plane, so
// most products take three instructions. (The fp32 matrix instructions run at a
// sixteenth of the bf16 rate: more than twice the time of six.)
//
// 16 x 16 x 32 instruction, lane = (m, g), m = lane % 16, g = lane / 16:
// operand A holds row m, B column m, 8 of the 32 inner indexes each; the result
// holds column m, rows 4 g to 4 g + 3. The inner index may run in any order that
// both operands share. Taken as "rows 4 g .. 4 g + 3 of the first tile of 16,
// then of the second", two results of one product are, lane by lane, an operand
// of the next: the state and the values of a chunk never leave registers. So that
// those rows are 8 neighbours in memory, tiles of dk and dv come in pairs of 32:
// row (or column) i of tile t is number delta_label(t, i).
#pragma once

#include "../layer/layer_common.h"

namespace pararnn {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ int delta_label(int t, int i) { return 32 * (t >> 1) + 8 * (i >> 2) + 4 * (t & 1) + (i & 3); }

// planes of a tensor of the caller. What is computed has three, also where the output that it goes to is bf16:
// with two of the state, P and y there, 16 bits, 3 in 1000 outputs fell to the other side of their rounding,
// for 4% of a prefill (B = 1 L = 65536 H = 16: 1220 us, 1170 with two)
template <class UT> struct DeltaPlanes { static constexpr int NP = 3; };
template <> struct DeltaPlanes<bf16> { static constexpr int NP = 1; };

// 8 fp32 values as N planes, each rounded to nearest
template <int N>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8* o) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int p = 0; p < N; ++p) {
    i32x4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = pack_bf16(r[2 * i], r[2 * i + 1]);
      u[i] = static_cast<int>(w);
      if (p + 1 < N) {
        r[2 * i] -= __uint_as_float(w << 16);
        r[2 * i + 1] -= __uint_as_float(w & 0xffff0000u);
      }
    }
    o[p] = __builtin_bit_cast(bf16x8, u);
  }
}
// two result tiles as an operand's block of 32
template <int N>
__device__ __forceinline__ void split_tiles(const f32x4& lo, const f32x4& hi, bf16x8* o) {
  const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  split8<N>(x, o);
}

// c[i] += a[i] b over their planes, the smallest products first (N: products of
// planes i and j with i + j < N); rows of a inside, so that no instruction waits
// for the one before it
template <int NA, int NB, int M>
__device__ __forceinline__ void mma_rows(f32x4 (&c)[M], const bf16x8 (&a)[M][NA], const bf16x8* b) {
  constexpr int N = NA > NB ? NA : NB;
#pragma unroll
  for (int s = N - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i <= s; ++i)
      if (i < NA && s - i < NB) {
#pragma unroll
        for (int r = 0; r < M; ++r) c[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[r][i], b[s - i], c[r], 0, 0, 0);
      }
}
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& c, const bf16x8* a, const bf16x8* b) {
  constexpr int N = NA > NB ? NA : NB;
#pragma unroll
  for (int s = N - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i <= s; ++i)
      if (i < NA && s - i < NB) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[s - i], c, 0, 0, 0);
}

// 8 consecutive elements of a row on their way from memory: loads through a
// buffer resource, without branches, so that they stay in flight until `planes`
// takes them. EVEN: every row starts at a multiple of 4 bytes (16-byte loads need
// no more); else bf16 elements come one by one.
template <class UT, bool EVEN>
struct Piece {
  static constexpr int N = sizeof(UT) == 4 ? 2 : 1;
  i32x4 v[N];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * i, 0, 0);
  }
  __device__ __forceinline__ uint32_t word(int i) const { return static_cast<uint32_t>(v[i >> 2][i & 3]); }
};
template <>
struct Piece<bf16, false> {
  uint16_t h[8];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = __builtin_amdgcn_raw_buffer_load_b16(r, off + 2 * i, 0, 0);
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    return static_cast<uint32_t>(h[2 * i]) | static_cast<uint32_t>(h[2 * i + 1]) << 16;
  }
};
// Sums of N values (a power of two) over LANES lanes that differ in the bits
// below `first`, dealt out: a step of the first log2(N) halves the values that a
// lane still has. Afterwards v[0] is the sum of value deal_index (of those bits).
template <int N, int LANES, int M>
__device__ __forceinline__ void sum_and_deal(float (&v)[M], int lane) {
  constexpr int OFF = LANES / 2;
  if constexpr (N > 1) {
    const bool up = (lane & OFF) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float send = up ? v[i] : v[i + N / 2], keep = up ? v[i + N / 2] : v[i];
      v[i] = keep + __shfl_xor(send, OFF, 64);
    }
  } else {
    v[0] += __shfl_xor(v[0], OFF, 64);
  }
  if constexpr (OFF > 1) sum_and_deal<(N > 1 ? N / 2 : 1), OFF>(v, lane);
}
// which of the N values a lane ends up with: the lanes' highest bits, in order
template <int N, int LANES>
__device__ __forceinline__ int deal_index(int lane) { return (lane & (LANES - 1)) / (LANES / N); }

// 4 x 4 values of 4 neighbouring lanes, transposed: lane q's v[c] becomes lane c's v[q]
template <int STEP>
__device__ __forceinline__ void swap_step(float& lo, float& hi, bool up) {
  const int send = __float_as_int(up ? lo : hi);
  const float got = __int_as_float(STEP == 1 ? __builtin_amdgcn_mov_dpp(send, 0xb1, 0xf, 0xf, true)    // lane ^ 1
                                             : __builtin_amdgcn_mov_dpp(send, 0x4e, 0xf, 0xf, true));  // lane ^ 2
  lo = up ? got : lo;
  hi = up ? hi : got;
}
__device__ __forceinline__ void transpose4(float (&v)[4], int lane) {
  swap_step<1>(v[0], v[1], lane & 1);
  swap_step<1>(v[2], v[3], lane & 1);
  swap_step<2>(v[0], v[2], lane & 2);
  swap_step<2>(v[1], v[3], lane & 2);
}

// How tensors come into workgroup memory: through registers (odd elements,
// 4-byte starts), or by 16-byte loads that write there (bf16 rows of whole chunks)
enum { kOdd = 0, kEven = 1, kDirect = 2 };
typedef __attribute__((address_space(3))) void lds_any;
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, void* to, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_any*)to, 16, off, 0, 0, 0);
}
constexpr uint32_t kNoLoad = 0x80000000u;  // past every resource's extent: reads zeros
// planes of the first `count` of a piece's elements, zeros behind them
template <class UT, bool EVEN>
__device__ __forceinline__ void planes_of(const Piece<UT, EVEN>& v, int count, bf16x8* o) {
  if constexpr (sizeof(UT) == 4) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < count ? __uint_as_float(v.word(i)) : 0.0f;
    split8<3>(x, o);
  } else {
    i32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = static_cast<int>(v.word(i) & (2 * i + 1 < count ? 0xffffffffu : 2 * i < count ? 0xffffu : 0u));
    o[0] = __builtin_bit_cast(bf16x8, w);
  }
}
template <int NP>
__device__ __forceinline__ float plane_sum(const bf16x8* o, int i) {
  float v = static_cast<float>(o[0][i]);
#pragma unroll
  for (int p = 1; p < NP; ++p) v += static_cast<float>(o[p][i]);
  return v;
}

template <class UT>
__device__ __forceinline__ float load1(const UT* p) {
  if constexpr (sizeof(UT) == 4) return *p;
  else return __uint_as_float(static_cast<uint32_t>(p->bits) << 16);
}
template <class UT>
__device__ __forceinline__ void store1(UT* p, float v) {
  if constexpr (sizeof(UT) == 4) *p = v;
  else p->bits = static_cast<uint16_t>(pack_bf16(v, v));
}
// the first `count` of 8 consecutive elements; wide: 16-byte aligned runs of 8
template <class UT>
__device__ __forceinline__ void store_run(UT* to, const float (&x)[8], int count, bool wide) {
  if (wide) {
    if constexpr (sizeof(UT) == 4) {
      *reinterpret_cast<f32x4*>(to) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4*>(to + 4) = f32x4{x[4], x[5], x[6], x[7]};
    } else {
      i32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = static_cast<int>(pack_bf16(x[2 * i], x[2 * i + 1]));
      *reinterpret_cast<i32x4*>(to) = v;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < count) store1(to + i, x[i]);
}

// A tile in workgroup memory: NP planes of ROWS rows of COLS bf16. Chunk c (16
// bytes) of a row lies at c ^ turn(row), so that 16 rows read at one chunk touch
// all banks, and 4 rows at 4 chunks as well.
template <int COLS, int NP, int ROWS = 64>
struct DeltaTile {
  static constexpr int CH = COLS / 8;  // chunks per row
  __bf16 x[NP][ROWS * COLS];
  static __device__ __forceinline__ int turn(int row) {
    return COLS >= 128 ? (row & 3) << 2 | (row >> 2 & 3) : COLS == 64 ? (row >> 1 & 1) << 2 | (row >> 2 & 3) : row >> 2 & 3;
  }
  static __device__ __forceinline__ int pos(int row, int col) {
    return row * COLS + (((col >> 3) ^ turn(row)) << 3) + (col & 7);
  }
  // operand A (rows) or B (columns): row 16 i + m, inner indexes the block kb of 32 columns
  __device__ __forceinline__ void rows(int i, int kb, int m, int g, bf16x8* o) const {
#pragma unroll
    for (int p = 0; p < NP; ++p)  // row 16 i + m has m's turn
      o[p] = *reinterpret_cast<const bf16x8*>(&x[p][(16 * i + m) * COLS + (((4 * kb + g) ^ turn(m)) << 3)]);
  }
  // the same of column m of tile t, inner indexes the block kb of 32 rows. Transposed reads: lane m of a group
  // gives the address of 4 columns of row m / 4 and gets 4 rows of column m.
  __device__ __forceinline__ void columns(int t, int kb, int m, int g, bf16x8* o) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int at = pos(32 * kb + 4 * g + (m >> 2), 32 * (t >> 1) + 8 * (m & 3) + 4 * (t & 1));  // 16 rows on: the same turn
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)&x[p][at]);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)&x[p][at + 16 * COLS]);
      o[p] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  // chunk number `slot` as the tile lies: row slot / CH, columns from source(slot) on
  static __device__ __forceinline__ int source(int slot) { return ((slot % CH) ^ turn(slot / CH)) << 3; }
  __device__ __forceinline__ void put_slot(int slot, const bf16x8* o) {
#pragma unroll
    for (int p = 0; p < NP; ++p) *reinterpret_cast<bf16x8*>(&x[p][slot * 8]) = o[p];
  }
  // 4 fp32 values at consecutive columns
  __device__ __forceinline__ void put4(int row, int col, const f32x4& v) {
    float r[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const uint32_t a = pack_bf16(r[0], r[1]), b = pack_bf16(r[2], r[3]);
      *reinterpret_cast<u32x2*>(&x[p][pos(row, col)]) = u32x2{a, b};
      r[0] -= __uint_as_float(a << 16);
      r[1] -= __uint_as_float(a & 0xffff0000u);
      r[2] -= __uint_as_float(b << 16);
      r[3] -= __uint_as_float(b & 0xffff0000u);
    }
  }
  __device__ __forceinline__ float at(int row, int col) const {
    const int i = pos(row, col);
    float v = static_cast<float>(x[0][i]);
#pragma unroll
    for (int p = 1; p < NP; ++p) v += static_cast<float>(x[p][i]);
    return v;
  }
};

}  // namespace pararnn
