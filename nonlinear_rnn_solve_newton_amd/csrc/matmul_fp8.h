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
// The 8-bit matrix instructions round the products that they add to about 2^-16
// of the largest (measured: 1.5e-5 of the result for Gaussian values, in the
// 16x16x128, 32x32x64 and 16x16x32 forms alike). That is far below the rounding
// of a bf16 result (2^-8). An fp32 result keeps its digits: its operands are
// widened to bf16, which holds every e4m3 value, and multiplied in that type,
// whose sums are good to 1e-8.
#pragma once

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

// one 16 x 16 tile of y^T over a whole 128-block, from zero
template <bool EXACT>
__device__ __forceinline__ f32x4 tile_product(const i32x8& w, const i32x8& a) {
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (EXACT) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8 x, y;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ws = w[2 * j + i], as = a[2 * j + i];
        const f32x2 w0 = __builtin_amdgcn_cvt_pk_f32_fp8(ws, false), w1 = __builtin_amdgcn_cvt_pk_f32_fp8(ws, true);
        const f32x2 a0 = __builtin_amdgcn_cvt_pk_f32_fp8(as, false), a1 = __builtin_amdgcn_cvt_pk_f32_fp8(as, true);
        x[4 * i] = static_cast<__bf16>(w0.x); x[4 * i + 1] = static_cast<__bf16>(w0.y);
        x[4 * i + 2] = static_cast<__bf16>(w1.x); x[4 * i + 3] = static_cast<__bf16>(w1.y);
        y[4 * i] = static_cast<__bf16>(a0.x); y[4 * i + 1] = static_cast<__bf16>(a0.y);
        y[4 * i + 2] = static_cast<__bf16>(a1.x); y[4 * i + 3] = static_cast<__bf16>(a1.y);
      }
      d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, d, 0, 0, 0);
    }
  } else {
    d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, d, 0, 0, 0, 127, 0, 127);
  }
  return d;
}

// 16 bytes of row `row` from column k on, zeros past the last column and row
__device__ __forceinline__ i32x4 load16(const uint8_t* p, long long row, int rows, int k, int K, bool aligned) {
  i32x4 v = {0, 0, 0, 0};
  if (row >= rows || k >= K) return v;
  const uint8_t* q = p + row * K + k;
  if (aligned) return *reinterpret_cast<const i32x4*>(q);
  uint8_t t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) t[i] = k + i < K ? q[i] : uint8_t{0};
  __builtin_memcpy(&v, t, 16);
  return v;
}

// 128 x 128 of y per workgroup of 4 waves, 64 x 64 per wave
constexpr int kTile = 128;
template <bool E8, bool EXACT, bool F32OUT>
__global__ void __launch_bounds__(256) matmul_kernel(const MatmulArgs p, int rows, int aligned) {
  __shared__ i32x4 s_w[kTile * 8], s_a[kTile * 8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int ntn = (p.N + kTile - 1) / kTile;
  const int m0 = static_cast<int>(blockIdx.x / ntn) * kTile, n0 = static_cast<int>(blockIdx.x % ntn) * kTile;
  const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
  f32x4 acc[4][4];  // [n][m]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = 0; kb < p.KB; ++kb) {
    __syncthreads();
    // 16-byte chunk c of row q lies at c ^ (q & 7): rows of 128 bytes read
    // down a column touch different banks
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid + 256 * i, q = e >> 3, c = e & 7;
      s_a[q * 8 + (c ^ (q & 7))] = load16(p.a, m0 + q, p.M, kb * 128 + c * 16, p.K, aligned);
      s_w[q * 8 + (c ^ (q & 7))] = load16(p.w, n0 + q, p.N, kb * 128 + c * 16, p.K, aligned);
    }
    __syncthreads();
    float sa[4];
    i32x8 fa[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = wm + 16 * j + r;
      sa[j] = scale_at<E8>(p.sa, static_cast<long long>(kb) * p.M + min(m0 + q, p.M - 1));
      const i32x4 lo = s_a[q * 8 + (g ^ (q & 7))], hi = s_a[q * 8 + ((g + 4) ^ (q & 7))];
      fa[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = wn + 16 * i + r;
      const i32x4 lo = s_w[q * 8 + (g ^ (q & 7))], hi = s_w[q * 8 + ((g + 4) ^ (q & 7))];
      const i32x8 fw = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      float sw[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int n = min(n0 + wn + 16 * i + 4 * g + v, p.N - 1);
        sw[v] = scale_at<E8>(p.sw, static_cast<long long>(rows == 1 ? n : n / 128) * p.KB + kb);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 d = tile_product<EXACT>(fw, fa[j]);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(d[v], sa[j] * sw[v], acc[i][j][v]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long m = m0 + wm + 16 * j + r;
      const int n = n0 + wn + 16 * i + 4 * g;
      if (m >= p.M) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (n + v >= p.N) continue;
        const float o = acc[i][j][v] + (p.bias ? p.bias[n + v] : 0.0f);
        if constexpr (F32OUT) static_cast<float*>(p.y)[m * p.N + n + v] = o;
        else static_cast<bf16*>(p.y)[m * p.N + n + v].bits = static_cast<uint16_t>(pack_bf16(o, o));
      }
    }
}

}  // namespace pararnn
