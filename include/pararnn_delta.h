/*
 * pararnn_delta.h -- C ABI of the operators of a delta-rule layer
 * (libpararnn_delta.so): a recurrence whose state is a matrix per head, next
 * to the vector states of pararnn_layer.h and pararnn.h.
 *
 * Conventions are those of pararnn_layer.h: device buffers that the caller
 * owns, scratch in the caller's workspace `ws` (256-byte aligned), calls
 * asynchronous on `stream`, status codes PARARNN_*, nothing launched on an
 * error other than PARARNN_EHIP, inputs and outputs that do not alias (except
 * where a call says "in place"). Sums, states and statistics are held in 32
 * bits; results are rounded once, to nearest even. Repeated calls give the
 * same bits. Sizes whose launch would have 2^32 threads or more are
 * PARARNN_EINVAL.
 */
#ifndef PARARNN_DELTA_H
#define PARARNN_DELTA_H

#include "pararnn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Gated delta rule. Per batch row b and value head v, whose q and k are those
 * of head v / (HV / H), with the state S [dk][dv]:
 *   q' = q / sqrt(|q|^2 + eps), k' = k / sqrt(|k|^2 + eps),
 *   log a = -c softplus(lam) s(gate_0), b = s(gate_1),      (s: logistic sigmoid)
 *   S_t = a S_{t-1} + k' b (v - a S_{t-1}^T k')^T,  S_{-1} = s0 (zero if NULL),
 *   o_t = scale S_t^T q'.
 */

/* A tensor [B][L][...] that is packed from its third dimension on, with the
 * elements between its rows and between its tokens: the columns of a wider
 * product are taken as they lie. Rows and tokens do not overlap. */
typedef struct {
  const void* p;
  int64_t batch, token; /* elements; token >= the packed size, batch >= L token (or B = 1) */
} pararnn_view;

typedef struct {
  int32_t B, L;             /* >= 1 */
  int32_t H, HV;            /* heads of q and k, heads of v: HV a multiple of H */
  int32_t dk, dv;           /* 1..128, 1..512 */
  int32_t dtype;            /* pararnn_dtype of q, k, v, gates, o and their gradients */
  float c, eps, scale;      /* c > 0, eps > 0, scale finite */
  const int32_t* lengths;   /* [B] (device) steps of each row, clamped to 0..L; NULL = L. Later steps leave the
                               state alone and put out zeros, whatever the inputs hold there */
  const uint8_t* reset;     /* [B][L] (device) nonzero: a document starts at this step, S_{t-1} counts as zero;
                               NULL = none */
} pararnn_delta_opts;

/* Workspace of pararnn_delta_scan (adjoint = 0) or _adjoint (adjoint = 1), and
 * bytes of `saved`, into *bytes. Host-only. */
int32_t pararnn_delta_workspace_bytes(int32_t adjoint, const pararnn_delta_opts* o, size_t* bytes);
int32_t pararnn_delta_saved_bytes(const pararnn_delta_opts* o, size_t* bytes);

/* Forward: q, k [B][L][H][dk], v [B][L][HV][dv], gates [B][L][2][HV] (decay,
 * write strength), lam [HV] fp32, s0 [B][HV][dk][dv] fp32 or NULL; o
 * [B][L][HV][dv], optionally sT [B][HV][dk][dv] fp32, the state after each
 * row's last step, and saved (256-byte aligned), what the adjoint starts from. */
int32_t pararnn_delta_scan(const pararnn_view* q, const pararnn_view* k, const pararnn_view* v,
                           const pararnn_view* gates, const float* lam, const float* s0, void* o, float* sT,
                           void* saved, void* ws, size_t ws_bytes, const pararnn_delta_opts* opts, void* stream);

/* Adjoint for d_o = dL/do [B][L][HV][dv] and, optionally, dsT = dL/dsT (NULL =
 * zero): dq, dk, dv and dgates, and optionally dlam (summed over B and L) and
 * ds0. Options as in the forward call that wrote `saved`. Gradients of steps
 * past a row's length are zero. */
int32_t pararnn_delta_scan_adjoint(const pararnn_view* q, const pararnn_view* k, const pararnn_view* v,
                                   const pararnn_view* gates, const float* lam, const void* saved, const void* d_o,
                                   const float* dsT, const pararnn_view* dq, const pararnn_view* dk,
                                   const pararnn_view* dv, const pararnn_view* dgates, float* dlam, float* ds0,
                                   void* ws, size_t ws_bytes, const pararnn_delta_opts* opts, void* stream);

/* One step for each of B requests (opts->L is 1, lengths and reset are not
 * used; a view's token stride is not either): q, k [B][H][dk], v [B][HV][dv],
 * gates [B][2][HV], o [B][HV][dv]; row b updates state[slots[b]] of the pool
 * state [S][HV][dk][dv] fp32 in place (NULL slots: state[b], S >= B). A slot
 * outside 0..S-1 is a row without a request: o = 0, no state touched. The slots
 * of one call must differ from each other. */
int32_t pararnn_delta_step(const pararnn_view* q, const pararnn_view* k, const pararnn_view* v,
                           const pararnn_view* gates, const float* lam, const int32_t* slots, float* state, void* o,
                           int32_t S, const pararnn_delta_opts* opts, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PARARNN_DELTA_H */
