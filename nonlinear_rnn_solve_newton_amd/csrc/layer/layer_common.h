// layer_common.h -- numerics and vector types shared by the kernels of the
// recurrent layer around the solver (gated_scan.h, norm.h, matmul_fp8.h).
// gfx950 (CDNA4) only.
#pragma once

#include "../device_common.h"

namespace pararnn {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// two fp32 values rounded to nearest even bf16, lo in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = __builtin_convertvector(f32x2{lo, hi}, bf16x2);
  return __builtin_bit_cast(uint32_t, v);
}

// C consecutive channels of type UT from fp32 registers through a buffer
// resource (stores past its extent are dropped)
template <class UT, int C, int AUX = 0>
__device__ __forceinline__ void buf_st(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, const float (&v)[C]) {
  if constexpr (sizeof(UT) == 4) {
    buf_st_f32<C, AUX>(r, voff, soff, v);
  } else if constexpr (C == 2) {
    __builtin_amdgcn_raw_buffer_store_b32(pack_bf16(v[0], v[1]), r, voff, soff, AUX);
  } else {
    __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(pack_bf16(v[0], v[0])), r, voff, soff, AUX);
  }
}

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|), to a few ulp for every x
// (also where it is tiny): the exponential's argument is split into two parts,
// and log1p(e) = 2 atanh(e / (2 + e)) by its series in s^2 <= 1/9, cut below
// 2^-26 of the sum.
__device__ __forceinline__ float softplus(float x) {
  const float ax = fabsf(x);
  const float y = ax * -1.4426950408889634f;
  const float lo = fmaf(ax, -1.4426950408889634f, -y) + ax * -1.925963033500e-8f;
  const float e = __builtin_amdgcn_exp2f(y);
  const float ec = fmaf(e * lo, 0.6931471805599453f, e);  // e 2^lo
  const float es = ax < 80.0f ? ec : e;                   // lo is not finite where x is not
  const float s = es * __builtin_amdgcn_rcpf(2.0f + es);
  const float q = s * s;
  float p = 1.0f / 15.0f;
  p = fmaf(p, q, 1.0f / 13.0f);
  p = fmaf(p, q, 1.0f / 11.0f);
  p = fmaf(p, q, 1.0f / 9.0f);
  p = fmaf(p, q, 1.0f / 7.0f);
  p = fmaf(p, q, 1.0f / 5.0f);
  p = fmaf(p, q, 1.0f / 3.0f);
  p = fmaf(p * q, 2.0f * s, 2.0f * s);
  return x != x ? x : fmaxf(x, 0.0f) + p;
}

}  // namespace pararnn
