/*
 * pararnn_layer.h -- C ABI of the operators of the recurrent layer around the
 * solver (libpararnn_layer.so): the norm in front of it, the 8-bit product
 * that makes its gate inputs, and the gated linear recurrence next to the
 * nonlinear cells of pararnn.h.
 *
 *   x, residual --norm_residual--> s (new residual), y (8 bits + scales)
 *   y, W --matmul_fp8--> u (gate inputs) --gated_scan / solve_gru / solve_lstm--> h
 *
 * Conventions are those of pararnn.h: contiguous row-major device buffers that
 * the caller owns, scratch in the caller's workspace `ws` (256-byte aligned),
 * calls asynchronous on `stream`, status codes PARARNN_*, nothing launched on
 * an error other than PARARNN_EHIP, inputs and outputs that do not alias
 * (except where a call says "in place"). Sums, states and statistics are held
 * in 32 bits; results are rounded once, to nearest even. Repeated calls give
 * the same bits. Sizes whose launch would have 2^32 threads or more (512 for
 * 32 or 64 channels of a row and 96 to 256 steps of a scan, one for 1 to 4
 * channels of a step, 256 or 512 for a tile of a product) are PARARNN_EINVAL.
 */
#ifndef PARARNN_LAYER_H
#define PARARNN_LAYER_H

#include "pararnn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Gated linear recurrence. Per batch row b and channel d, gates (r, i, x):
 *   r = s(u_r), i = s(u_i), log a = -c softplus(lam) r, a = exp(log a),
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,   h_{-1} = h0 (zero if NULL).
 * Layouts: u [B][L][3][D], h, dh [B][L][D], du [B][L][3][D] in `dtype`;
 * lam, dlam [D], h0, hT, dh0, dhT [B][D] fp32.
 */
typedef struct {
  int32_t B, L, D;          /* all >= 1 */
  int32_t dtype;            /* pararnn_dtype of u, h, dh and du */
  float c;                  /* > 0 and finite */
  const int32_t* lengths;   /* [B] (device) steps of each row, clamped to 0..L; NULL = L.
                               Later steps leave the state alone and put out h = 0, du = 0,
                               whatever u and dh hold there */
  const uint8_t* reset;     /* [B][L] (device) nonzero: a document starts at this step, h_{t-1}
                               counts as zero; NULL = none */
} pararnn_gated_opts;

/* Workspace of pararnn_gated_scan (adjoint = 0) or _adjoint (adjoint = 1) into
 * *bytes, enough with and without lengths and reset; it may be 0, and ws then
 * NULL. Host-only. */
int32_t pararnn_gated_workspace_bytes(int32_t adjoint, const pararnn_gated_opts* o, size_t* bytes);

/* Number of saved states per channel: one in front of every 96 steps. */
int32_t pararnn_gated_saved_rows(int32_t L);

/* Forward: h, and optionally hT, the state after each row's last step, and
 * saved [saved_rows(L)][B][D] fp32, the states the adjoint starts from (those
 * past a row's length may stay unwritten). */
int32_t pararnn_gated_scan(const void* u, const float* lam, const float* h0, void* h, float* hT, float* saved,
                           void* ws, size_t ws_bytes, const pararnn_gated_opts* o, void* stream);

/* Adjoint for dh = dL/dh and, optionally, dhT = dL/dhT (NULL = zero): du, and
 * optionally dlam (summed over B and L) and dh0. Options as in the forward
 * call that wrote `saved`. */
int32_t pararnn_gated_scan_adjoint(const void* u, const float* lam, const float* saved, const void* dh,
                                   const float* dhT, void* du, float* dlam, float* dh0, void* ws, size_t ws_bytes,
                                   const pararnn_gated_opts* o, void* stream);

/* One step for each of B requests: u [B][3][D], h [B][D] in `dtype`; row b
 * updates state[slots[b]] of the pool state [S][D] fp32 in place (NULL slots:
 * state[b], S >= B). A slot outside 0..S-1 is a row without a request: h = 0,
 * no state touched. The slots of one call must differ from each other. */
int32_t pararnn_gated_step(const void* u, const float* lam, const int32_t* slots, float* state, void* h, int32_t B,
                           int32_t D, int32_t S, int32_t dtype, float c, void* stream);

/* ---------------------------------------------------------------------------
 * Root-mean-square norm with the residual's addition, rows of D columns:
 *   s = x + residual (x if NULL),  y = s / sqrt(mean(s^2) + eps) * w.
 * x, residual, s, dy, ds, dx [N][D] in `dtype`, w, dw [D] fp32.
 */
typedef enum {
  PARARNN_NORM_SAME = 0,      /* y [N][D] in `dtype`; scale is not used */
  PARARNN_NORM_FP8 = 1,       /* y [N][D] e4m3, scale [ceil(D/128)][N] fp32 */
  PARARNN_NORM_FP8_E8M0 = 2   /* y [N][D] e4m3, scale [ceil(D/128)][N] e8m0 (powers of two) */
} pararnn_norm_out;

typedef struct {
  int64_t N;      /* rows, >= 1 */
  int32_t D;      /* columns, 1..16384 */
  int32_t dtype;  /* pararnn_dtype */
  int32_t out;    /* pararnn_norm_out; ignored by the adjoint */
  float eps;      /* >= 0 and finite */
} pararnn_norm_opts;

/* Forward: y, and optionally s (NULL: not written), from one pass. y is made
 * from the sum before its rounding to `dtype`. With an 8-bit y every 128
 * columns of a row share scale = max(max|y|, 2^-100) / 448, or the next power
 * of two at or above that, and hold y / scale (the fp32 quotient) rounded to
 * nearest even; a block with an infinity or a NaN stands for NaN. */
int32_t pararnn_norm_residual(const void* x, const void* residual, const float* w, void* s, void* y, void* scale,
                              const pararnn_norm_opts* o, void* stream);

/* Workspace of the adjoint's dw; 0 for invalid options. Host-only. */
size_t pararnn_norm_workspace_bytes(const pararnn_norm_opts* o);

/* Adjoint for dy = dL/dy and, optionally, ds = dL/ds of the other uses of s
 * (NULL = zero): dx (the gradient of x and of the residual), and optionally
 * dw (NULL: not computed, and no workspace needed). An 8-bit y passes its
 * gradient straight through. */
int32_t pararnn_norm_residual_adjoint(const void* s, const float* w, const void* dy, const void* ds, void* dx,
                                      float* dw, void* ws, size_t ws_bytes, const pararnn_norm_opts* o,
                                      void* stream);

/* ---------------------------------------------------------------------------
 * Product of 8-bit (e4m3) matrices with a scale for each block of 128 along K:
 *   y[m][n] = sum_k a[m][k] sa[k/128][m] w[n][k] sw[n/w_rows][k/128] + bias[n].
 * a [M][K], sa [ceil(K/128)][M] (as norm_residual writes them), w [N][K],
 * sw [ceil(N/w_rows)][ceil(K/128)], bias [N] fp32 or NULL, y [M][N].
 * With N = G*D this makes the gate inputs u [B*L][G][D] of the recurrences.
 * A bf16 y is computed with the 8-bit matrix instructions, which cut products to
 * multiples of 2^-13 of the power of two of the largest of eight neighbours
 * (along k) before they add them in fp32: at most 2^-10.2 of the sum of the
 * products' magnitudes, 1e-6 to 1e-5 of it for operands of one size. An fp32 y
 * comes from exact products. Scales whose product is below 2^-126 or 2^128 and
 * above are outside what the scaling in fp32 holds. K % 16 == 0 with 16-byte
 * aligned a and w selects the widest accesses.
 */
typedef enum { PARARNN_SCALE_F32 = 0, PARARNN_SCALE_E8M0 = 1 } pararnn_scale_type;

typedef struct {
  int32_t M, N, K;   /* all >= 1; K <= 2^22 */
  int32_t w_rows;    /* rows of w that share a scale: 128 or 1 */
  int32_t scale;     /* pararnn_scale_type of sa and sw */
  int32_t y_dtype;   /* pararnn_dtype of y */
} pararnn_matmul_opts;

int32_t pararnn_matmul_fp8(const void* a, const void* sa, const void* w, const void* sw, const float* bias, void* y,
                           const pararnn_matmul_opts* o, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PARARNN_LAYER_H */
