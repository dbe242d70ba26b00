// norm_block.h -- the norms before and after a block of a layer, with the gate
// and the residual's scale between them, and their adjoint. Over rows of D
// columns (s: logistic sigmoid):
//   n = x / sqrt(mean(x^2) + eps) w        over groups of G columns (x itself without w)
//   p = n gate s(gate)                      (n without a gate)
//   r = residual + alpha p,  y = r / sqrt(mean(r^2) + eps) w_next;  without a residual y = p
//   8 bits: per row scale = max(max|y|, 2^-100) / 127, q = round(y / scale).
// Adjoint, with xh = x rstd, rh = r rstd_r, c = gate s(gate), and dr the whole gradient of r:
//   t = dy w_next,  dr = rstd_r (t - rh mean(t rh)) + ds,  dp = alpha dr  (dp = dy without a residual)
//   dgate = dp n s(gate) (1 + gate (1 - s(gate))),  u = dp c w,  dx = rstd (u - xh mean(u xh))
//   dw = sum of dp c xh,  dalpha = sum of dr p,  dw_next = sum of dy rh  over rows (and groups).
//
// One pass over the row: it stays in registers, 8 consecutive columns per lane
// and vector, NV vectors, so each tensor crosses HBM once. Groups without a
// residual are rows of their own (w is theirs, and so are the threads of a
// wave's part); groups beside a residual, or whose 8-bit scale is the row's,
// are parts of a wave: G / 8 lanes. HBM bounds many rows: 32768 x 1024 in groups of 128
// with a gate, bf16, 32 to 35 us (201 MB, 5.7 to 6.3 TB/s) and 57 us for the adjoint (336
// MB, 5.9); 32768 x 4096 with a residual to 8 bits 163 us (5.6 TB/s). Few rows are the
// latency of a load, two sums and a store: 16 x 4096 5.3 us. The adjoint's parameters
// take a sum over the workgroups' partial rows in a launch of its own (5 us).
#pragma once

#include "delta_common.h"

namespace pararnn {

struct NormBlockArgs {
  const void *x, *gate, *residual;  // gate, residual: or nullptr
  const float *w, *alpha, *w_next;  // or nullptr
  void *s, *y;                      // s: r in the input's type; y: the input's type or int8
  float* scale;                     // [N] with 8 bits
  const void *dy, *ds;              // adjoint: residual is the saved r; ds: or nullptr
  void *dx, *dgate, *dresidual;
  float* part;                      // adjoint: [gridDim.x][3][D] sums of dw, dalpha, dw_next, or nullptr
  long long N, x_row, gate_row, residual_row;  // rows; elements from row to row of the inputs
  int D, H;    // columns; rows per row of memory: row n lies at (n / H) x_row + (n % H) D
  int lanes;   // lanes per group (a power of two up to 64), 0: the row is the group
  int G;       // columns of w
  float eps;
};

// 8 consecutive columns from d on of a row of D; aligned: every row is a whole
// number of 16-byte accesses. Else rows start at any element and take 16 bytes
// wherever 8 columns are left (unaligned accesses are what the device is set to).
template <class XT, bool ALIGNED, bool STREAM>
struct Vec8 {
  i32x4 v[sizeof(XT) / 2];
  __device__ __forceinline__ void load(const XT* p, int d, int D) {
    constexpr int N = sizeof(XT) / 2, E = 16 / sizeof(XT);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = i32x4{0, 0, 0, 0};
      const XT* q = p + d + E * i;
      if constexpr (ALIGNED) {
        if (d < D) {
          if constexpr (STREAM) v[i] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(q));
          else v[i] = *reinterpret_cast<const i32x4*>(q);
        }
      } else if (d + E * (i + 1) <= D) {
        __builtin_memcpy(&v[i], q, 16);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (d + E * i + e < D) {
            if constexpr (sizeof(XT) == 4) v[i][e] = __float_as_int(q[e]);
            else v[i][e / 2] |= static_cast<int>(static_cast<uint32_t>(q[e].bits) << (16 * (e & 1)));
          }
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(XT) == 4) return __int_as_float(v[i >> 2][i & 3]);
    else return i & 1 ? bf16_hi(static_cast<uint32_t>(v[0][i >> 1])) : bf16_lo(static_cast<uint32_t>(v[0][i >> 1]));
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(XT) == 4) {
        v[0][i] = __float_as_int(x[i]);
        v[1][i] = __float_as_int(x[4 + i]);
      } else {
        v[0][i] = static_cast<int>(pack_bf16(x[2 * i], x[2 * i + 1]));
      }
    }
  }
  __device__ __forceinline__ void store(XT* p, int d, int D) const {
    constexpr int N = sizeof(XT) / 2, E = 16 / sizeof(XT);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      XT* q = p + d + E * i;
      if constexpr (ALIGNED) {
        if (d < D) {
          if constexpr (STREAM) __builtin_nontemporal_store(v[i], reinterpret_cast<i32x4*>(q));
          else *reinterpret_cast<i32x4*>(q) = v[i];
        }
      } else if (d + E * (i + 1) <= D) {
        __builtin_memcpy(q, &v[i], 16);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (d + E * i + e < D) {
            if constexpr (sizeof(XT) == 4) q[e] = __int_as_float(v[i][e]);
            else q[e].bits = static_cast<uint16_t>(static_cast<uint32_t>(v[i][e / 2]) >> (16 * (e & 1)));
          }
      }
    }
  }
};
// 8 columns of an fp32 parameter of D columns; ones where there is none
template <bool ALIGNED>
__device__ __forceinline__ void load_param(const float* w, int d, int D, float (&v)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    return;
  }
  Vec8<float, ALIGNED, false> x;
  x.load(w, d, D);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x.at(i);
}

// sum (MAX: largest) of NS values over the TPR threads of a row, in a fixed order; every thread gets it
template <int TPR, int NS, bool MAX = false>
__device__ __forceinline__ void over_row(float (&v)[NS], float* lds, int tid) {
#pragma unroll
  for (int off = (TPR < 64 ? TPR : 64) / 2; off >= 1; off >>= 1)
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const float u = __shfl_xor(v[k], off, 64);
      v[k] = MAX ? fmaxf(v[k], u) : v[k] + u;
    }
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64, ALL = (TPR < 256 ? 256 : TPR) / 64;  // waves of a row, of the workgroup
    __syncthreads();  // the sums before these have been read
    if ((tid & 63) == 0) {
#pragma unroll
      for (int k = 0; k < NS; ++k) lds[k * ALL + (tid >> 6)] = v[k];
    }
    __syncthreads();
    const float* row = lds + tid / TPR * W;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      v[k] = row[k * ALL];
#pragma unroll
      for (int w = 1; w < W; ++w) v[k] = MAX ? fmaxf(v[k], row[k * ALL + w]) : v[k] + row[k * ALL + w];
    }
  }
}
// the same within groups of `lanes` lanes
template <int NS>
__device__ __forceinline__ void over_lanes(float (&v)[NS], int lanes) {
  for (int off = lanes >> 1; off >= 1; off >>= 1)
#pragma unroll
    for (int k = 0; k < NS; ++k) v[k] += __shfl_xor(v[k], off, 64);
}
__device__ __forceinline__ long long row_at(long long row, int H, long long stride, int D) {
  return H == 1 ? row * stride : row / H * stride + row % H * D;
}

// A workgroup takes BT / TPR rows at a time. PRE: with a residual.
template <class XT, int TPR, int NV, bool PRE, bool INT8, bool ALIGNED, bool STREAM>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_block_kernel(const NormBlockArgs p) {
  constexpr int BT = TPR < 256 ? 256 : TPR, RW = BT / TPR;
  typedef Vec8<XT, ALIGNED, STREAM> V;
  __shared__ float lds[2 * (BT / 64)];
  const int tid = threadIdx.x, t = tid % TPR, rw = tid / TPR;
  const float inv_g = 1.0f / static_cast<float>(p.lanes ? p.G : p.D), inv_d = 1.0f / static_cast<float>(p.D);
  float wv[NV][8], al[PRE ? NV : 1][8], wn[PRE ? NV : 1][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int d = 8 * (t + TPR * k);
    load_param<ALIGNED>(p.w, p.lanes ? d % p.G : d, p.lanes ? p.G : p.D, wv[k]);
    if constexpr (PRE) {
      load_param<ALIGNED>(p.alpha, d, p.D, al[k]);
      load_param<ALIGNED>(p.w_next, d, p.D, wn[k]);
    }
  }
  // every wave of a workgroup runs the same number of rounds
  for (long long row0 = static_cast<long long>(blockIdx.x) * RW; row0 < p.N; row0 += static_cast<long long>(gridDim.x) * RW) {
    const bool on = row0 + rw < p.N;
    const long long row = on ? row0 + rw : 0, out = row * p.D;
    V x[NV], z[NV], r[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int d = 8 * (t + TPR * k);
      x[k].load(static_cast<const XT*>(p.x) + row_at(row, p.H, p.x_row, p.D), d, p.D);
      if (p.gate) z[k].load(static_cast<const XT*>(p.gate) + row_at(row, p.H, p.gate_row, p.D), d, p.D);
      if constexpr (PRE) r[k].load(static_cast<const XT*>(p.residual) + row * p.residual_row, d, p.D);
    }
    float v[NV][8];
    float one[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float q[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[k][i] = x[k].at(i);
        q[0] = fmaf(v[k][i], v[k][i], q[0]);
      }
      if (p.lanes) {
        over_lanes<1>(q, p.lanes);
        const float rstd = 1.0f / sqrtf(fmaf(q[0], inv_g, p.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] *= rstd;
      } else {
        one[0] += q[0];
      }
    }
    if (p.w && !p.lanes) {
      over_row<TPR, 1>(one, lds, tid);
      const float rstd = 1.0f / sqrtf(fmaf(one[0], inv_g, p.eps));
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] *= rstd;
    }
    float sum[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int d = 8 * (t + TPR * k);
      if (p.w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] *= wv[k][i];
      }
      if (p.gate) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] *= z[k].at(i) * sigm(z[k].at(i));
      }
      if constexpr (PRE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[k][i] = fmaf(al[k][i], v[k][i], r[k].at(i));
          sum[0] = fmaf(v[k][i], v[k][i], sum[0]);
        }
        if (on) {
          r[k].set(v[k]);
          r[k].store(static_cast<XT*>(p.s) + out, d, p.D);
        }
      }
    }
    if constexpr (PRE) {
      over_row<TPR, 1>(sum, lds, tid);
      const float rstd = 1.0f / sqrtf(fmaf(sum[0], inv_d, p.eps));
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] *= rstd * wn[k][i];
    }
    if constexpr (!INT8) {
      if (on) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          x[k].set(v[k]);
          x[k].store(static_cast<XT*>(p.y) + out, 8 * (t + TPR * k), p.D);
        }
      }
    } else {
      // the row's largest magnitude; a NaN anywhere makes it NaN, and the row then stands for NaN
      float big[2] = {0x1p-100f, 0.0f};
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * (t + TPR * k) + i < p.D) {
            big[0] = fmaxf(big[0], fabsf(v[k][i]));
            big[1] = v[k][i] != v[k][i] ? 1.0f : big[1];
          }
      over_row<TPR, 2, true>(big, lds, tid);
      const float scale = big[1] != 0.0f ? __uint_as_float(0x7fc00000u) : big[0] / 127.0f, inv = 1.0f / scale;
      if (on && t == 0) p.scale[row] = scale;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int d = 8 * (t + TPR * k);
        int q[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // the quotient, correctly rounded: the product with the inverse and its remainder's
          float u = v[k][i] * inv;
          u = fmaf(fmaf(-u, scale, v[k][i]), inv, u);
          u = fminf(fmaxf(u, -127.0f), 127.0f);  // NaN: some number, times a scale that is NaN or infinite
          q[i >> 2] |= (static_cast<int>(rintf(u)) & 255) << (8 * (i & 3));
        }
        int8_t* to = static_cast<int8_t*>(p.y) + out + d;
        if (on && d < p.D) {
          if (ALIGNED) {
            *reinterpret_cast<i32x2*>(to) = i32x2{q[0], q[1]};
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (d + i < p.D) to[i] = static_cast<int8_t>(q[i >> 2] >> (8 * (i & 3)));
          }
        }
      }
    }
  }
}

// Gradients per row; those of the parameters summed in registers over the
// workgroup's rows, one partial row of each per workgroup for norm_block_sum_kernel
template <class XT, int TPR, int NV, bool PRE, bool ALIGNED, bool STREAM>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_block_adjoint_kernel(const NormBlockArgs p) {
  constexpr int BT = TPR < 256 ? 256 : TPR, RW = BT / TPR, NP = PRE ? 3 : 1;
  typedef Vec8<XT, ALIGNED, STREAM> V;
  __shared__ float lds[3 * (BT / 64)];
  __shared__ float fold[RW > 1 ? RW : 1][RW > 1 ? TPR * NV * 8 : 1];
  const int tid = threadIdx.x, t = tid % TPR, rw = tid / TPR;
  const float inv_g = 1.0f / static_cast<float>(p.lanes ? p.G : p.D), inv_d = 1.0f / static_cast<float>(p.D);
  // The parameters are held over the rows, or, where a thread has 16 columns or 128 registers, read anew for every
  // row (4096 x 8192 with a residual, 512 threads: 126 us, held 241; 4096 x 4096, one vector: 71, held 66)
  constexpr bool HOLD = TPR * NV <= 512;
  constexpr int NH = HOLD ? NV : 1;
  const float *pw = p.w, *pa = p.alpha, *pn = p.w_next;
  float wv[NH][8], al[PRE ? NH : 1][8], wn[PRE ? NH : 1][8], part[NP][NV][8];
  auto load_w = [&](int k, float (&v)[8]) {
    const int d = 8 * (t + TPR * k);
    load_param<ALIGNED>(pw, p.lanes ? d % p.G : d, p.lanes ? p.G : p.D, v);
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      load_w(k, wv[k]);
      if constexpr (PRE) {
        load_param<ALIGNED>(pa, 8 * (t + TPR * k), p.D, al[k]);
        load_param<ALIGNED>(pn, 8 * (t + TPR * k), p.D, wn[k]);
      }
    }
  }
#pragma unroll
  for (int a = 0; a < NP; ++a)
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) part[a][k][i] = 0.0f;
  for (long long row0 = static_cast<long long>(blockIdx.x) * RW; row0 < p.N; row0 += static_cast<long long>(gridDim.x) * RW) {
    const bool on = row0 + rw < p.N;
    const long long row = on ? row0 + rw : 0, out = row * p.D;
    if constexpr (!HOLD) __asm__ volatile("" : "+s"(pw), "+s"(pa), "+s"(pn));  // not before the loop
    V x[NV], z[NV], s[NV], dy[NV], ds[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int d = 8 * (t + TPR * k);
      x[k].load(static_cast<const XT*>(p.x) + row_at(row, p.H, p.x_row, p.D), d, p.D);
      dy[k].load(static_cast<const XT*>(p.dy) + out, d, p.D);
      if (p.gate) z[k].load(static_cast<const XT*>(p.gate) + row_at(row, p.H, p.gate_row, p.D), d, p.D);
      if constexpr (PRE) {
        s[k].load(static_cast<const XT*>(p.residual) + out, d, p.D);
        if (p.ds) ds[k].load(static_cast<const XT*>(p.ds) + out, d, p.D);
      }
    }
    // sums of the whole row: x^2, r^2, t r
    float sum[3] = {0.0f, 0.0f, 0.0f}, rstd[NV], u[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float q[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i) q[0] = fmaf(x[k].at(i), x[k].at(i), q[0]);
      if (p.lanes) {
        over_lanes<1>(q, p.lanes);
        rstd[k] = 1.0f / sqrtf(fmaf(q[0], inv_g, p.eps));
      }
      sum[0] += q[0];
      if constexpr (PRE) {
        if constexpr (!HOLD) load_param<ALIGNED>(pn, 8 * (t + TPR * k), p.D, wn[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float r = s[k].at(i);
          u[k][i] = dy[k].at(i) * wn[HOLD ? k : 0][i];
          sum[1] = fmaf(r, r, sum[1]);
          sum[2] = fmaf(u[k][i], r, sum[2]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[k][i] = dy[k].at(i);
      }
    }
    if (PRE || !p.lanes) over_row<TPR, 3>(sum, lds, tid);
    if (!p.lanes) {
      const float r0 = p.w ? 1.0f / sqrtf(fmaf(sum[0], inv_g, p.eps)) : 1.0f;
#pragma unroll
      for (int k = 0; k < NV; ++k) rstd[k] = r0;
    }
    const float rr = 1.0f / sqrtf(fmaf(sum[1], inv_d, p.eps)), mean = sum[2] * rr * inv_d;
    float dot[1] = {0.0f}, dots[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int d = 8 * (t + TPR * k);
      float g[8];
      if constexpr (PRE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float rh = s[k].at(i) * rr;
          if (on) part[2][k][i] = fmaf(dy[k].at(i), rh, part[2][k][i]);
          u[k][i] = fmaf(rr, fmaf(-rh, mean, u[k][i]), p.ds ? ds[k].at(i) : 0.0f);  // dr
        }
        if (on) {
          s[k].set(u[k]);
          s[k].store(static_cast<XT*>(p.dresidual) + out, d, p.D);
        }
      }
      float q = 0.0f;
      if constexpr (!HOLD) {
        load_w(k, wv[0]);
        if constexpr (PRE) load_param<ALIGNED>(pa, d, p.D, al[0]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = x[k].at(i) * rstd[k], n = xh * wv[HOLD ? k : 0][i];
        float c = 1.0f, dc = 0.0f;
        if (p.gate) {
          const float zi = z[k].at(i), sz = sigm(zi);
          c = zi * sz;
          dc = sz * fmaf(zi, 1.0f - sz, 1.0f);
        }
        if constexpr (PRE) {
          if (on) part[1][k][i] = fmaf(u[k][i], n * c, part[1][k][i]);
          u[k][i] *= al[HOLD ? k : 0][i];
        }
        g[i] = u[k][i] * n * dc;
        const float v = u[k][i] * c;
        if (on) part[0][k][i] = fmaf(v, xh, part[0][k][i]);
        u[k][i] = v * wv[HOLD ? k : 0][i];
        q = fmaf(u[k][i], xh, q);
      }
      if (p.gate && on) {
        z[k].set(g);
        z[k].store(static_cast<XT*>(p.dgate) + out, d, p.D);
      }
      if (p.lanes) {
        float one[1] = {q};
        over_lanes<1>(one, p.lanes);
        dots[k] = one[0];
      }
      dot[0] += q;
    }
    if (!p.lanes && p.w) over_row<TPR, 1>(dot, lds, tid);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const float m = p.w ? (p.lanes ? dots[k] : dot[0]) * inv_g : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) u[k][i] = rstd[k] * fmaf(-(x[k].at(i) * rstd[k]), m, u[k][i]);
      if (on) {
        x[k].set(u[k]);
        x[k].store(static_cast<XT*>(p.dx) + out, 8 * (t + TPR * k), p.D);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int a = 0; a < NP; ++a) {
    float* to = p.part + (static_cast<long long>(blockIdx.x) * NP + a) * p.D;
    if constexpr (RW > 1) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) fold[rw][8 * (t + TPR * k) + i] = part[a][k][i];
      __syncthreads();
      for (int d = tid; d < p.D; d += BT) {
        float v = fold[0][d];
#pragma unroll
        for (int r = 1; r < RW; ++r) v += fold[r][d];
        to[d] = v;
      }
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * (t + TPR * k) + i < p.D) to[8 * (t + TPR * k) + i] = part[a][k][i];
    }
  }
}

// Sums of the partial rows, in a fixed order: workgroup (j, a) takes 32 columns
// of output a. w's columns of groups beside each other fold into one.
__global__ void __launch_bounds__(1024)
norm_block_sum_kernel(const float* part, float* dw, float* dalpha, float* dw_next, long long rows, int NP, int D, int G) {
  __shared__ float s[32][33];
  const int j = threadIdx.x & 31, q = threadIdx.x >> 5, a = blockIdx.y, col = blockIdx.x * 32 + j;
  float* out = a == 0 ? dw : a == 1 ? dalpha : dw_next;
  const int cols = a == 0 ? G : D, fold = D / cols;
  float acc = 0.0f;
  if (out && col < cols) {
    for (int h = 0; h < fold; ++h) {
      const float* at = part + static_cast<long long>(a) * D + h * cols + col;
      const long long step = static_cast<long long>(NP) * D;
      long long r = q;
      for (; r + 3 * 32 < rows; r += 4 * 32) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = at[(r + 32 * i) * step];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc += v[i];
      }
      for (; r < rows; r += 32) acc += at[r * step];
    }
  }
  s[q][j] = acc;
  __syncthreads();
  if (q == 0 && out && col < cols) {
    float v = 0.0f;
    for (int k = 0; k < 32; ++k) v += s[k][j];
    out[col] = v;
  }
}

}  // namespace pararnn
