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
 * the same bits.
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

/* Workspace of pararnn_gated_scan (adjoint = 0) or _adjoint (adjoint = 1);
 * 0 for invalid options. Host-only. */
size_t pararnn_gated_workspace_bytes(int32_t adjoint, const pararnn_gated_opts* o);

/* Number of saved states per channel: one in front of every 128 steps. */
int32_t pararnn_gated_saved_rows(int32_t L);

/* Forward: h, and optionally hT, the state after each row's last step, and
 * saved [saved_rows(L)][B][D] fp32, the states the adjoint starts from. */
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

#ifdef __cplusplus
}
#endif

#endif /* PARARNN_LAYER_H */
