/*
 * twell_lm.h -- the operators that stand around the activation-sparse FFN in
 * a language model (same library, libtwell.so; one GB300, sm_103a):
 *
 *   token ids -> twell_embed_* -> twell_add_rmsnorm_* -> twell_ffn_* -> ...
 *     -> twell_add_rmsnorm_* -> output product -> twell_distill_*   (training)
 *     -> twell_add_rmsnorm_* (8-bit output) -> twell_q8_matmul      (serving)
 *
 * The conventions of twell.h hold for every call: device pointers owned by
 * the caller, asynchronous on `stream`, errors the host can see are returned
 * before anything is launched, no allocation, scratch (256-byte aligned) from
 * the caller.  What only the device can see goes to the caller's `status`
 * word (device int32, 0 before the first call, the first error wins;
 * twell_read_status reads and clears it).  Row-major contiguous operands
 * unless a row pitch is given; pointers 16-byte aligned except the per-row
 * and per-column vectors, which take their type's own alignment (the norm's
 * weight 16 bytes, a pair of stats 8).  Operands, stream and current device are
 * one GPU's, the same for all calls of a process.  Element
 * type `dtype`: TWELL_F32 or TWELL_BF16.  Sums, maxima, statistics and norms
 * are held in fp32 (8-bit products: exact in fp32, see twell_q8_matmul), each
 * output is rounded once (to nearest even), and every result is independent
 * of scheduling: the same call gives the same bits.  Numbers of tokens, rows
 * and output columns are at most 2^30 (element offsets are 64-bit throughout);
 * sizes beyond what an entry states return TWELL_ERR_ARG.
 */
#ifndef TWELL_LM_H
#define TWELL_LM_H

#include "twell.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Synchronise `stream`, read and clear a status word; returns it, or
 * TWELL_ERR_CUDA. */
twell_status twell_read_status(int32_t *status, void *stream);

/* ---- token embedding ------------------------------------------------------
 * out[t] = scale * table[token t]            table [V][D], out [T][D], dtype
 * tokens [T]: int32 (token_bytes 4) or int64 (8).  A position whose token is
 * pad_id gives a zero row and takes no gradient (pad_id = -1 pads nothing but
 * -1).  Any other token outside [0, V) is treated the same way and records
 * TWELL_ERR_INDEX.  1 <= T, 1 <= V < 2^31 - 1, D <= 65536; D*elem_size a
 * multiple of 16. */
twell_status twell_embed_forward(const void *tokens, int token_bytes, const void *table, int T,
                                 int V, int D, int dtype, float scale, long long pad_id,
                                 void *out, int32_t *status, void *stream);

/* dtable[v] = scale * sum over the positions t with token v of dy[t], in
 * ascending t (fixed grouping of the fp32 sum); rows of tokens that do not
 * occur are written 0.  dy [T][D] dtype; dtable [V][D] fp32, overwritten.
 * The tokens are sorted on the device (stable); nothing uses floating-point
 * atomics. */
twell_status twell_embed_backward(const void *tokens, int token_bytes, const void *dy, int T,
                                  int V, int D, int dtype, float scale, long long pad_id,
                                  float *dtable, int32_t *status, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* Scratch bytes of twell_embed_backward (0 for invalid sizes). */
size_t twell_embed_workspace_size(int T, int V, int D);

/* ---- residual addition + root-mean-square norm ------------------------------
 * s = x + residual (residual may be NULL: s = x), stored in dtype
 * rstd = 1 / sqrt(mean(s^2) + eps),  y = s * rstd * weight
 * The norm reads the stored s, so that the backward, which has only s, is
 * the gradient of exactly this function.
 *   x, residual, s, y [T][D] dtype; weight [D] fp32; rstd [T] fp32
 *   s may be NULL when residual is NULL, and may be the same buffer as x or
 *   residual.  Any of y, q (with qscale) and rstd may be NULL, but not both
 *   y and q.
 * 8-bit output: q [T][D] int8, qscale [T] fp32: qscale = max|y| / 127 over
 * the row, q = y / qscale rounded to nearest even, so y ~ q * qscale (y in
 * fp32, not rounded to dtype first).  A row of zeros has qscale 0; a row with
 * an infinity or NaN has q 0 and qscale NaN.  A finite row whose mean(s^2) + eps
 * leaves the normal fp32 range, upwards or (with eps below 2^-126, 0 among them)
 * downwards, as a row of zeros does, has rstd 0, y 0, q 0 and qscale 0.
 * 16 <= D*elem_size <= 16384, a multiple of 16 (TWELL_BF16 with q: D a
 * multiple of 16). */
twell_status twell_add_rmsnorm_forward(const void *x, const void *residual, const float *weight,
                                       int T, int D, int dtype, float eps, void *s, void *y,
                                       int8_t *q, float *qscale, float *rstd, void *stream);

/* xhat = s * rstd
 * dx = ds + rstd * (weight*dy - xhat * mean(weight*dy*xhat))
 * dweight = sum over rows of dy * xhat   (fp32, overwritten)
 * dx is the gradient of x and of the residual alike; ds [T][D] (the gradient
 * that reaches s past the norm) may be NULL, and dx may be the same buffer as
 * ds or dy. */
twell_status twell_add_rmsnorm_backward(const void *s, const float *weight, const float *rstd,
                                        const void *dy, const void *ds, int T, int D, int dtype,
                                        void *dx, float *dweight, void *workspace,
                                        size_t workspace_bytes, void *stream);

/* Scratch bytes of twell_add_rmsnorm_backward (0 for invalid sizes). */
size_t twell_add_rmsnorm_workspace_size(int T, int D);

/* ---- 8-bit product -----------------------------------------------------------
 * Symmetric 8-bit rows of a matrix: scale[r] = max|a[r]| / 127, q = a / scale
 * rounded to nearest even (zero and non-finite rows as in the norm's 8-bit
 * output).  For weights, once; rows >= 1, cols*elem_size and cols multiples
 * of 16. */
twell_status twell_q8_quantize(const void *a, int rows, int cols, int dtype, int8_t *q,
                               float *scale, void *stream);

/* y[m][n] = ascale[m] * wscale[n] * sum_k aq[m][k] wq[n][k]  (+ bias[n])
 *   aq [M][K], wq [N][K] int8 (the full range, -128 included), ascale [M],
 *   wscale [N], bias [N] or NULL: fp32; y [M][N] dtype.
 * K a multiple of 16, 16 <= K <= 65536; 1 <= M, N.  The integer sum is exact
 * while its partial sums stay below 2^24 in magnitude (always for K <= 1024)
 * and otherwise a sum in fp32. */
twell_status twell_q8_matmul(const int8_t *aq, const float *ascale, const int8_t *wq,
                             const float *wscale, const float *bias, int M, int N, int K,
                             int dtype, void *y, int32_t *status, void *workspace,
                             size_t workspace_bytes, void *stream);

/* Scratch bytes of twell_q8_matmul (0 for invalid sizes). */
size_t twell_q8_workspace_size(int M, int N, int K);

/* ---- distillation from a teacher's top logits ---------------------------------
 * z [T][V] (row pitch ldz elements) dtype: the student's logits.
 * ids, teacher [T][k]: the teacher's top entries (token id, fp32 logit); an
 * id < 0 marks an unused entry, an id >= V records TWELL_ERR_INDEX and is not
 * used.  An id that occurs twice counts with both probabilities.
 *   p = softmax(teacher / tau) over the row's entries
 *   q = softmax(z / tau) over the vocabulary
 *   loss[t] = row_weight[t] * tau^2 * sum_i p_i (log p_i - log q_{id_i})
 *   dz[t]   = row_weight[t] * tau * (q - p)
 *   stats[t] = {max z, log sum exp((z - max z) / tau)}   (for the backward)
 * row_weight [T] fp32, NULL: all 1.  A row of weight 0 is not read: its loss,
 * stats and dz are 0.  A row without entries has loss 0 and dz 0.  Logits of
 * -inf (and of the type's lowest value beside larger ones) have q = 0; a row
 * with NaN, +inf or nothing but -inf has loss and dz NaN.
 * dz (NULL: not computed) has z's type and pitch and may be z itself; with
 * it, loss and gradient take one pass over the logits.
 * 1 <= T, 1 <= V <= ldz, 1 <= k <= 256, 1e-4 <= tau <= 1e4. */
twell_status twell_distill_forward(const void *z, long long ldz, const int32_t *ids,
                                   const float *teacher, const float *row_weight, int T, int V,
                                   int k, int dtype, float tau, float *loss, float *stats,
                                   void *dz, int32_t *status, void *stream);

/* dz[t] = row_grad[t] * tau * (q - p) from the forward's stats: row_grad =
 * row_weight * (gradient that reaches the row's loss).  Rows of row_grad 0
 * are not read and get 0.  dz may be z itself. */
twell_status twell_distill_backward(const void *z, long long ldz, const int32_t *ids,
                                    const float *teacher, const float *stats,
                                    const float *row_grad, int T, int V, int k, int dtype,
                                    float tau, void *dz, int32_t *status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TWELL_LM_H */
