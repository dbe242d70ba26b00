// norm.h -- root-mean-square norm with the residual's addition, written in the
// input's type or in 8 bits with a scale for each 128 columns, and its adjoint.
//   s = x + residual,   rstd = 1 / sqrt(mean(s^2) + eps),   y = s rstd w
//   8 bits (e4m3): per row and 128 columns, scale = max(max|y|, 2^-100) / 448
//   (or the next power of two at or above that), q = round(y / scale), the
//   quotient rounded to fp32 first.
// Adjoint, with t = dy w and n = s rstd:
//   dx = rstd (t - n mean(t n)) + ds,   dw = sum over rows of dy n.
//
// One pass over the row: it stays in registers (8 consecutive columns per lane
// and vector, NV vectors) between the sum of squares and the output, so each
// tensor crosses HBM once. Bound by HBM: 32768 x 4096 bf16 with a residual to 8
// bits takes 160 us (5.9 TB/s), its adjoint to bf16 197 us (5.4 TB/s); 4999 x
// 1000, which the caches hold, 9.1 us and 11.8 + 4.5 us (the sum of dw's
// partial rows), 16 x 4096 4.2 us, all of it latency.
#pragma once

#include "layer_common.h"

namespace pararnn {

enum { kNormSame = 0, kNormFp8 = 1, kNormFp8Pow2 = 2 };
constexpr float kE4m3Max = 448.0f;

struct NormArgs {
  const void* x;         // [N][D]
  const void* residual;  // [N][D] or nullptr
  const float* w;        // [D]
  void* s;               // [N][D] or nullptr
  void* y;               // [N][D]: the input's type or e4m3
  void* scale;           // [ceil(D / 128)][N] fp32 or e8m0; nullptr unless 8 bits
  const void* dy;        // adjoint: x is s
  const void* ds;        // [N][D] or nullptr
  void* dx;
  float* dw_part;        // [gridDim.x][D] or nullptr
  long long N;
  int D;
  float eps;
};

// STREAM: past the caches
template <bool STREAM, class V>
__device__ __forceinline__ V ld_vec(const V* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool STREAM, class V>
__device__ __forceinline__ void st_vec(V* p, V v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}
// 8 consecutive columns starting at d: one wide access where every row is
// aligned for it (VEC), else single elements up to D; columns past D read 0
template <class XT, bool VEC, bool STREAM = false>
__device__ __forceinline__ void ld8(const XT* p, int d, int D, float (&v)[8]) {
  if constexpr (VEC) {
    if (d < D) {
      if constexpr (sizeof(XT) == 4) {
        const f32x4 a = ld_vec<STREAM>(reinterpret_cast<const f32x4*>(p + d));
        const f32x4 b = ld_vec<STREAM>(reinterpret_cast<const f32x4*>(p + d + 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
      } else {
        const i32x4 a = ld_vec<STREAM>(reinterpret_cast<const i32x4*>(p + d));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = bf16_lo(static_cast<uint32_t>(a[i]));
          v[2 * i + 1] = bf16_hi(static_cast<uint32_t>(a[i]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(XT) == 4) v[i] = d + i < D ? p[d + i] : 0.0f;
      else v[i] = d + i < D ? __uint_as_float(static_cast<uint32_t>(p[d + i].bits) << 16) : 0.0f;
    }
  }
}
template <class XT, bool VEC, bool STREAM>
__device__ __forceinline__ void st8(XT* p, int d, int D, const float (&v)[8]) {
  if constexpr (VEC) {
    if (d < D) {
      if constexpr (sizeof(XT) == 4) {
        st_vec<STREAM>(reinterpret_cast<f32x4*>(p + d), f32x4{v[0], v[1], v[2], v[3]});
        st_vec<STREAM>(reinterpret_cast<f32x4*>(p + d + 4), f32x4{v[4], v[5], v[6], v[7]});
      } else {
        i32x4 a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = static_cast<int>(pack_bf16(v[2 * i], v[2 * i + 1]));
        st_vec<STREAM>(reinterpret_cast<i32x4*>(p + d), a);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d + i < D) {
        if constexpr (sizeof(XT) == 4) p[d + i] = v[i];
        else p[d + i].bits = static_cast<uint16_t>(pack_bf16(v[i], v[i]));
      }
  }
}

// sum of NS values over the TPR threads of a row, in a fixed order; every
// thread gets it
template <int TPR, int NS>
__device__ __forceinline__ void row_sum(float (&v)[NS], float* lds, int tid) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1)
#pragma unroll
    for (int k = 0; k < NS; ++k) v[k] += __shfl_xor(v[k], off, 64);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    __syncthreads();  // the previous row's sums have been read
    if ((tid & 63) == 0) {
#pragma unroll
      for (int k = 0; k < NS; ++k) lds[k * W + (tid >> 6)] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      v[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[k] += lds[k * W + w];
    }
  }
}

// A workgroup takes 256 / TPR rows at a time (1 where TPR is 256 or more); OUT: kNorm*
template <class XT, int TPR, int NV, int OUT, bool VEC, bool STREAM>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_kernel(const NormArgs p) {
  constexpr int BT = TPR < 256 ? 256 : TPR, RW = BT / TPR;
  __shared__ float s_sum[BT / 64];
  const int tid = threadIdx.x, t = tid % TPR, rw = tid / TPR;
  float wv[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) ld8<float, VEC>(p.w, 8 * (t + TPR * k), p.D, wv[k]);
  const float inv_d = 1.0f / static_cast<float>(p.D);
  // every wave of a workgroup runs the same number of rounds
  for (long long row0 = static_cast<long long>(blockIdx.x) * RW; row0 < p.N; row0 += static_cast<long long>(gridDim.x) * RW) {
    const long long row = row0 + rw;
    const bool on = row < p.N;
    const long long at = (on ? row : 0) * p.D;
    float s[NV][8];
    float ss[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k) ld8<XT, VEC, STREAM>(static_cast<const XT*>(p.x) + at, 8 * (t + TPR * k), p.D, s[k]);
    if (p.residual) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float r[8];
        ld8<XT, VEC, STREAM>(static_cast<const XT*>(p.residual) + at, 8 * (t + TPR * k), p.D, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[k][i] += r[i];
      }
    }
    if (p.s && on) {
#pragma unroll
      for (int k = 0; k < NV; ++k) st8<XT, VEC, STREAM>(static_cast<XT*>(p.s) + at, 8 * (t + TPR * k), p.D, s[k]);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = fmaf(s[k][i], s[k][i], ss[0]);
    row_sum<TPR, 1>(ss, s_sum, tid);
    const float rstd = 1.0f / sqrtf(fmaf(ss[0], inv_d, p.eps));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int d = 8 * (t + TPR * k);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[k][i] = s[k][i] * rstd * wv[k][i];
      if constexpr (OUT == kNormSame) {
        if (on) st8<XT, VEC, STREAM>(static_cast<XT*>(p.y) + at, d, p.D, s[k]);
      } else {
        // the block's largest magnitude, by bits: a NaN counts as the largest
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(s[k][i]) & 0x7fffffffu);
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), off, 64)));
        m = max(m, 0x0d800000u);  // 2^-100
        const float scale = __uint_as_float(m) / kE4m3Max;
        float inv;
        const long long si = static_cast<long long>(d / 128) * p.N + row;
        if constexpr (OUT == kNormFp8) {
          inv = 1.0f / scale;
          if (on && (t & 15) == 0 && d < p.D) static_cast<float*>(p.scale)[si] = scale;
        } else {
          const uint32_t sb = __float_as_uint(scale);
          const uint32_t e = min((sb >> 23) + ((sb & 0x7fffffu) ? 1u : 0u), 255u);
          inv = e == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((254u - e) << 23);
          if (on && (t & 15) == 0 && d < p.D) static_cast<uint8_t*>(p.scale)[si] = static_cast<uint8_t>(e);
        }
        // the quotients by scale, correctly rounded: by a power of two the product with its inverse, else
        // that product and its remainder's (two fused operations per element, free next to HBM)
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = s[k][i] * inv;
          if constexpr (OUT == kNormFp8) v[i] = fmaf(fmaf(-v[i], scale, s[k][i]), inv, v[i]);
        }
        int q0 = 0, q1 = 0;
        q0 = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], q0, false);
        q0 = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], q0, true);
        q1 = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], q1, false);
        q1 = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], q1, true);
        uint8_t* q = static_cast<uint8_t*>(p.y) + at + d;
        if constexpr (VEC) {
          if (on && d < p.D) st_vec<STREAM>(reinterpret_cast<i32x2*>(q), i32x2{q0, q1});
        } else if (on) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (d + i < p.D) q[i] = static_cast<uint8_t>((i < 4 ? q0 : q1) >> (8 * (i & 3)));
        }
      }
    }
  }
}

// dx per row; dw summed in registers over the workgroup's rows, one partial
// row per workgroup for column_sum_kernel
template <class XT, int TPR, int NV, bool VEC, bool STREAM>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_adjoint_kernel(const NormArgs p) {
  constexpr int BT = TPR < 256 ? 256 : TPR, RW = BT / TPR;
  __shared__ float s_sum[2 * (BT / 64)];
  __shared__ float s_dw[RW > 1 ? RW : 1][RW > 1 ? TPR * NV * 8 : 1];
  const int tid = threadIdx.x, t = tid % TPR, rw = tid / TPR;
  float wv[NV][8], dw[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    ld8<float, VEC>(p.w, 8 * (t + TPR * k), p.D, wv[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = 0.0f;
  }
  const float inv_d = 1.0f / static_cast<float>(p.D);
  for (long long row0 = static_cast<long long>(blockIdx.x) * RW; row0 < p.N; row0 += static_cast<long long>(gridDim.x) * RW) {
    const long long row = row0 + rw;
    const bool on = row < p.N;
    const long long at = (on ? row : 0) * p.D;
    float s[NV][8], g[NV][8];
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      ld8<XT, VEC, STREAM>(static_cast<const XT*>(p.x) + at, 8 * (t + TPR * k), p.D, s[k]);
      ld8<XT, VEC, STREAM>(static_cast<const XT*>(p.dy) + at, 8 * (t + TPR * k), p.D, g[k]);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0] = fmaf(s[k][i], s[k][i], sum[0]);
        sum[1] = fmaf(g[k][i] * wv[k][i], s[k][i], sum[1]);
      }
    row_sum<TPR, 2>(sum, s_sum, tid);
    const float rstd = 1.0f / sqrtf(fmaf(sum[0], inv_d, p.eps));
    const float mean = sum[1] * rstd * inv_d;  // of t n
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int d = 8 * (t + TPR * k);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = 0.0f;
      if (p.ds) ld8<XT, VEC, STREAM>(static_cast<const XT*>(p.ds) + at, d, p.D, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = s[k][i] * rstd;
        o[i] = fmaf(rstd, fmaf(-n, mean, g[k][i] * wv[k][i]), o[i]);
        if (on) dw[k][i] = fmaf(g[k][i], n, dw[k][i]);
      }
      if (on) st8<XT, VEC, STREAM>(static_cast<XT*>(p.dx) + at, d, p.D, o);
    }
  }
  if (!p.dw_part) return;
  float* part = p.dw_part + static_cast<long long>(blockIdx.x) * p.D;
  if constexpr (RW > 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s_dw[rw][8 * (t + TPR * k) + i] = dw[k][i];
    __syncthreads();
    for (int d = tid; d < p.D; d += BT) {
      float v = s_dw[0][d];
#pragma unroll
      for (int r = 1; r < RW; ++r) v += s_dw[r][d];
      part[d] = v;
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int d = 8 * (t + TPR * k);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (d + i < p.D) part[d + i] = dw[k][i];
    }
  }
}

}  // namespace pararnn
