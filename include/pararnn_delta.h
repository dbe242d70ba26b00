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
 * bits, those that go to bf16 outputs too; results are rounded once, to
 * nearest even. Squares are summed in fp32: |q|^2, |k|^2 and the squares of a
 * normed row must not pass its largest number. Repeated calls give the
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
  int64_t batch, token; /* elements; token from the packed size to 2^22, batch from (L - 1) token + the packed size
                           to 2^50 (or B = 1) */
} pararnn_view;

typedef struct {
  int32_t B, L;             /* >= 1 */
  int32_t H, HV;            /* heads of q and k, heads of v: HV a multiple of H */
  int32_t dk, dv;           /* 1..128, 1..512 */
  int32_t dtype;            /* pararnn_dtype of q, k, v, gates, o and their gradients */
  float c, eps, scale;      /* c > 0, eps > 0, scale finite */
  const int32_t* lengths;   /* [B] (device) steps of each row, clamped to 0..L; NULL = L. Later steps leave the
                               state alone and put out zeros, whatever the inputs hold there or before */
  const uint8_t* reset;     /* [B][L] (device) nonzero: a document starts at this step, S_{t-1} counts as zero;
                               NULL = none. (An infinity or a NaN among a row's steps reaches, in its heads, the
                               steps after it, over a start too, and none in front of it; in the adjoint all of the
                               row's.) */
} pararnn_delta_opts;

/* Workspace of pararnn_delta_scan (adjoint = 0) or _adjoint (adjoint = 1), and
 * bytes of `saved`, into *bytes. Host-only. Of each value head and 64 steps,
 * with dk and dv up to the next multiples of 32, `saved` takes 4 dv (dk + 64)
 * bytes (96 KB at 128 x 128), the workspace 39 KB, and in the adjoint as much as
 * `saved` besides; few heads add their segments' matrices, up to 32 MB. */
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

/* ---------------------------------------------------------------------------
 * Norms before and after a block, with the gate and the residual's scale
 * between them, over rows of D columns:
 *   n = x / sqrt(mean(x^2) + eps) * w  over groups of `group` columns (x without w),
 *   p = n * gate * s(gate)  (n without a gate),
 *   s = residual + alpha * p,  y = s / sqrt(mean(s^2) + eps) * w_next;
 *   without a residual (and then without alpha, w_next and s): y = p.
 * x, gate, residual, dy, ds, dx, dgate, dresidual [N][D] in `dtype`; w, dw
 * [group], alpha, dalpha, w_next, dw_next [D] fp32. w or a residual is given.
 */
typedef enum {
  PARARNN_NORM_BLOCK_SAME = 0, /* y [N][D] in `dtype` */
  PARARNN_NORM_BLOCK_INT8 = 1  /* y [N][D] int8, scale [N] fp32 */
} pararnn_norm_block_out;

typedef struct {
  int64_t N;       /* rows, >= 1 */
  int32_t D;       /* columns, 1..16384 */
  int32_t group;   /* columns of a group of x, a divisor of D. Groups of less than D beside a residual or an
                      8-bit y are 8, 16, 32, ... 512 columns */
  int32_t dtype;   /* pararnn_dtype */
  int32_t out;     /* pararnn_norm_block_out; ignored by the adjoint */
  float eps;       /* >= 0 and finite */
  int64_t x_row, gate_row, residual_row; /* elements from row to row of those inputs, >= D; the adjoint's s has D */
} pararnn_norm_block_opts;

/* Forward: y, and s with a residual. y is made from the sum before its
 * rounding to `dtype`. An 8-bit row has scale = max(max|y|, 2^-100) / 127 and
 * holds y / scale (the fp32 quotient) rounded to nearest even; a row with an
 * infinity or a NaN has a scale that is infinite or NaN and stands for no
 * numbers. */
int32_t pararnn_norm_block(const void* x, const void* gate, const void* residual, const float* w, const float* alpha,
                           const float* w_next, void* s, void* y, float* scale, const pararnn_norm_block_opts* o,
                           void* stream);

/* Workspace of the adjoint's dw, dalpha and dw_next into *bytes. Host-only. */
int32_t pararnn_norm_block_workspace_bytes(const pararnn_norm_block_opts* o, int32_t residual, size_t* bytes);

/* Adjoint for dy = dL/dy and, with a residual, ds = dL/ds of the other uses of
 * s (NULL = zero), at the saved s (NULL: the forward call had no residual): dx,
 * dgate (with a gate), dresidual (with a residual), and, all of them optional,
 * dw, dalpha and dw_next (all NULL: no workspace needed). An 8-bit y passes its
 * gradient straight through. */
int32_t pararnn_norm_block_adjoint(const void* x, const void* gate, const void* s, const float* w, const float* alpha,
                                   const float* w_next, const void* dy, const void* ds, void* dx, void* dgate,
                                   void* dresidual, float* dw, float* dalpha, float* dw_next, void* ws,
                                   size_t ws_bytes, const pararnn_norm_block_opts* o, void* stream);

/* ---------------------------------------------------------------------------
 * Product of 8-bit integer matrices with a scale for each row of both:
 *   y[m][n] = sum_k a[m][k] w[n][k] * sa[m] * sw[n] + bias[n].
 * a [M][K], sa [M] fp32 (as norm_block writes them), w [N][K], sw [N] fp32,
 * bias [N] fp32 or NULL, y [M][N]. The sum is exact (32-bit integers); it is
 * rounded to fp32 once, and the rest is computed in fp32. K % 16 == 0 with
 * 16-byte aligned a and w selects the widest accesses.
 */
typedef struct {
  int32_t M, N, K; /* all >= 1; K <= 131071 (whose sum of products of -128 still fits) */
  int32_t y_dtype; /* pararnn_dtype of y */
} pararnn_int8_opts;

int32_t pararnn_matmul_int8(const void* a, const float* sa, const void* w, const float* sw, const float* bias, void* y,
                            const pararnn_int8_opts* o, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PARARNN_DELTA_H */
