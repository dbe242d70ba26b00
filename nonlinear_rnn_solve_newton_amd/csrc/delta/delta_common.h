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
// of the next: the state and the values of a chunk never leave registers.
#pragma once

#include "../layer/layer_common.h"

namespace pararnn {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// planes of a tensor of the caller (NP), and those that an output of its type
// needs of an fp32 factor (NO: 16 bits below bf16's own rounding of 8)
template <class UT> struct DeltaPlanes { static constexpr int NP = 3, NO = 3; };
template <> struct DeltaPlanes<bf16> { static constexpr int NP = 1, NO = 2; };

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

// c += a b over their planes, the smallest products first; PB: planes of b that
// count, N: the order kept (products of planes i and j with i + j < N)
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& c, const bf16x8* a, const bf16x8* b) {
  constexpr int N = NA > NB ? NA : NB;
#pragma unroll
  for (int s = N - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i <= s; ++i)
      if (i < NA && s - i < NB) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[s - i], c, 0, 0, 0);
}

// 8 consecutive elements as they lie in memory
template <class UT> struct Raw8 {
  f32x4 a, b;
  __device__ __forceinline__ float at(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
};
template <> struct Raw8<bf16> {
  i32x4 a;
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = static_cast<uint32_t>(a[i >> 1]);
    return i & 1 ? bf16_hi(w) : bf16_lo(w);
  }
};
// elements d .. d + 7 of a row of n; zeros past its end and where `on` is false. wide: the row's start and n
// are multiples of 16 bytes and of 8.
template <class UT>
__device__ __forceinline__ Raw8<UT> load_raw8(const UT* row, int d, int n, bool on, bool wide) {
  Raw8<UT> v = {};
  if (!on || d >= n) return v;
  if (wide) {
    if constexpr (sizeof(UT) == 4) {
      v.a = *reinterpret_cast<const f32x4*>(row + d);
      v.b = *reinterpret_cast<const f32x4*>(row + d + 4);
    } else {
      v.a = *reinterpret_cast<const i32x4*>(row + d);
    }
    return v;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (d + i < n) {
      if constexpr (sizeof(UT) == 4) {
        if (i < 4) v.a[i & 3] = row[d + i];
        else v.b[i & 3] = row[d + i];
      } else {
        v.a[i >> 1] |= static_cast<int>(static_cast<uint32_t>(row[d + i].bits) << (16 * (i & 1)));
      }
    }
  return v;
}
// planes of 8 elements of the caller's type
__device__ __forceinline__ void planes_of(const Raw8<bf16>& v, bf16x8* o) { o[0] = __builtin_bit_cast(bf16x8, v.a); }
__device__ __forceinline__ void planes_of(const Raw8<float>& v, bf16x8* o) {
  const float x[8] = {v.a[0], v.a[1], v.a[2], v.a[3], v.b[0], v.b[1], v.b[2], v.b[3]};
  split8<3>(x, o);
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
// 8 consecutive elements of a row of n from d on
template <class UT>
__device__ __forceinline__ void store8(UT* row, int d, int n, bool wide, const float (&x)[8]) {
  if (d >= n) return;
  if (wide) {
    if constexpr (sizeof(UT) == 4) {
      *reinterpret_cast<f32x4*>(row + d) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4*>(row + d + 4) = f32x4{x[4], x[5], x[6], x[7]};
    } else {
      i32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = static_cast<int>(pack_bf16(x[2 * i], x[2 * i + 1]));
      *reinterpret_cast<i32x4*>(row + d) = v;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (d + i < n) store1(row + d + i, x[i]);
}

// A chunk's rows of q or k in workgroup memory: NP planes of 64 rows, 16
// elements longer than DK, so that both ways of reading them are spread over
// the banks.
template <int DK, int NP>
struct DeltaTile {
  static constexpr int ROW = DK + 16;
  __bf16 x[NP][64 * ROW];
  // operand A, rows of the chunk: row 16 i + m, inner indexes of the block kb of 32 columns
  __device__ __forceinline__ void rows(int i, int kb, int m, int g, bf16x8* o) const {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const __bf16* at = &x[p][(16 * i + m) * ROW + 32 * kb + 4 * g];
      const u32x2 lo = *reinterpret_cast<const u32x2*>(at), hi = *reinterpret_cast<const u32x2*>(at + 16);
      o[p] = __builtin_bit_cast(bf16x8, i32x4{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(hi.x),
                                              static_cast<int>(hi.y)});
    }
  }
  // operand A (rows) or B (columns): column 16 t + m, inner indexes the rows of the block kb of 32. Transposed
  // reads: lane m of a group gives the address of 4 columns of row m / 4 and gets 4 rows of column m.
  __device__ __forceinline__ void columns(int t, int kb, int m, int g, bf16x8* o) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      __bf16* at = &x[p][(32 * kb + 4 * g + (m >> 2)) * ROW + 16 * t + 4 * (m & 3)];
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * ROW));
      o[p] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  template <class UT>
  __device__ __forceinline__ void put(int row, int d, const Raw8<UT>& v) {
    bf16x8 o[NP];
    planes_of(v, o);
#pragma unroll
    for (int p = 0; p < NP; ++p) *reinterpret_cast<bf16x8*>(&x[p][row * ROW + d]) = o[p];
  }
  __device__ __forceinline__ float at(int row, int d) const {
    float v = static_cast<float>(x[0][row * ROW + d]);
#pragma unroll
    for (int p = 1; p < NP; ++p) v += static_cast<float>(x[p][row * ROW + d]);
    return v;
  }
};

}  // namespace pararnn
