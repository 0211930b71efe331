/*
 * twell_lm.h -- the operators that stand around the activation-sparse FFN in
 * a language model (same library, libtwell.so; one GB300, sm_103a):
 *
 *   token ids -> twell_embed_* -> twell_add_rmsnorm_* -> twell_recur_*
 *     -> twell_add_rmsnorm_* -> twell_ffn_* -> ...
 *     -> twell_add_rmsnorm_* -> output product
 *          -> twell_distill_* or twell_policy_*, back, twell_adamw_step (training)
 *     -> twell_add_rmsnorm_* (8-bit output) -> twell_q8_matmul        (serving)
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

/* ---- gated linear recurrence over packed sequences ------------------------------
 * a_t = sigmoid(gate_t + bias),  c_t = 1 - a_t   (channel by channel)
 * h_t = a_t h_{t-1} + c_t x_t,   h_{-1} = h0 of the sequence
 *   x, gate [T][D] dtype, row pitch ld elements (the halves of one projection's
 *   rows, or matrices of their own); bias [D] fp32 or NULL; h [T][D] dtype.
 *   starts [B + 1] int32 on the device, ascending: sequence s is the rows
 *   starts[s] .. starts[s + 1] - 1 (none: an empty sequence).  Rows before the
 *   first and behind the last sequence are not read, and their outputs are left
 *   as they were.  starts NULL: B sequences of T / B rows each.  Values that
 *   descend or leave [0, T] record TWELL_ERR_INDEX; the outputs are then undefined.
 *   h0 [B][D] fp32: the states before the sequences (NULL: 0); hT [B][D] fp32 or
 *   NULL: the states behind them (of an empty sequence: h0).  hT may be h0.
 *   states [twell_recur_states(T)][D] fp32 or NULL: what the backward needs.
 * The state is held in fp32, h is its rounding; h is a buffer of its own.  B = T
 * without starts is the step of a decoded token for each of T sequences.
 * a and c are each right to 2^-15 of themselves, the small one beside 1 included: a
 * state that gates have forgotten leaves nothing.  Where x, h0, dh or dhT is infinite
 * or NaN, or h - x beyond fp32's range, what depends on it by these formulas is infinite
 * or NaN (h from that row of its sequence on, G up to it), and nothing else.
 * 1 <= T, 1 <= B, D <= 65536, D <= ld <= 2^34; D*elem_size and ld*elem_size multiples
 * of 16. */
twell_status twell_recur_forward(const void *x, const void *gate, long long ld, const float *bias,
                                 const int32_t *starts, int B, const float *h0, int T, int D,
                                 int dtype, void *h, float *hT, float *states, int32_t *status,
                                 void *stream);

/* G_t = dh_t + a_{t+1} G_{t+1} within the sequence (a_{t+1} G_{t+1} = dhT at its last row)
 * dx = c G,  dgate = G (h_{t-1} - x) a c,  dbias = sum over rows of dgate
 * dh0 = a G at the sequence's first row (an empty sequence: dhT)
 *   dh [T][D] dtype, dhT [B][D] fp32 (NULL: 0); dx, dgate [T][D] dtype, row pitch
 *   ld; dbias [D] and dh0 [B][D] fp32, overwritten, each may be NULL.
 * x, gate, bias, starts, h0 and states as in the forward (whose fp32 states the
 * backward takes up again, so that h and its rounding do not matter).  The outputs
 * may not be the inputs' buffers. */
twell_status twell_recur_backward(const void *x, const void *gate, long long ld,
                                  const float *bias, const int32_t *starts, int B,
                                  const float *h0, const float *states, const void *dh,
                                  const float *dhT, int T, int D, int dtype, void *dx,
                                  void *dgate, float *dbias, float *dh0, int32_t *status,
                                  void *stream);

/* Rows of `states` (0 for an invalid T). */
int twell_recur_states(int T);

/* ---- clipped policy loss with a KL term -----------------------------------------
 * z [T][V] (row pitch ldz elements) dtype: the policy's logits.  tokens [T] int32
 * (token_bytes 4) or int64 (8): the sampled ones.
 *   logp = z[token] / tau - log sum exp(z / tau)
 *   r = exp(logp - old_logp)       (old_logp NULL: old_logp = logp, r = 1)
 *   d = ref_logp - logp            (ref_logp NULL: no KL term)
 *   loss[t] = row_weight[t] * (-min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
 *                              + beta (exp(d) - d - 1)),  A = advantage[t]
 *   slope   = row_weight[t] * (-(r A, or 0 where the clipped side is the smaller)
 *                              + beta (1 - exp(d)))        d loss / d logp
 *   dz[t]   = slope / tau * (onehot(token) - softmax(z / tau))
 *   stats[t] = {max z, log sum exp((z - max z) / tau)}
 * old_logp, ref_logp, advantage, row_weight (NULL: all 1), loss, logp [T] fp32.
 * A row of weight 0 or with a token < 0 is not read: its loss, logp, stats and dz
 * are 0.  A token >= V records TWELL_ERR_INDEX, and its row is treated the same.
 * Logits of -inf have probability 0; a row with NaN, +inf or nothing but -inf has
 * loss, logp and dz NaN (with advantage 0 and no KL term: loss and dz 0 or NaN).  A
 * token of probability 0 has logp -inf: r is 0 and, with beta > 0, the loss infinite
 * (old_logp and ref_logp finite).  The terms of the slope, and row_weight * slope / tau,
 * are held within +-2^126, which exp(d) reaches near d = 87, so that dz is finite there
 * too, and 0 at other elements of probability 0.
 * advantage NULL: the log-probabilities alone (loss and dz NULL), as for old_logp
 * and ref_logp themselves.  dz (else NULL: not computed) has z's type and pitch and
 * may be z itself.
 * 1 <= T, 1 <= V <= ldz, 1e-4 <= tau <= 1e4, 0 <= clip_low <= 1, 0 <= clip_high,
 * 0 <= beta, all finite. */
twell_status twell_policy_forward(const void *z, long long ldz, const void *tokens,
                                  int token_bytes, const float *old_logp, const float *ref_logp,
                                  const float *advantage, const float *row_weight, int T, int V,
                                  int dtype, float tau, float clip_low, float clip_high,
                                  float beta, float *loss, float *logp, float *stats, void *dz,
                                  int32_t *status, void *stream);

/* dz from the forward's logp and stats; row_grad in the place of row_weight:
 * row_weight * (gradient that reaches the row's loss).  dz may be z itself. */
twell_status twell_policy_backward(const void *z, long long ldz, const void *tokens,
                                   int token_bytes, const float *old_logp, const float *ref_logp,
                                   const float *advantage, const float *logp, const float *stats,
                                   const float *row_grad, int T, int V, int dtype, float tau,
                                   float clip_low, float clip_high, float beta, void *dz,
                                   int32_t *status, void *stream);

/* ---- AdamW over many tensors ------------------------------------------------------
 * For every element of every tensor, with g = grad (* *grad_scale):
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   param = param (1 - lr decay)
 *           - lr / correction1 * m / (sqrt(v) / sqrt(correction2) + eps)
 *   copy = param in bf16 (where there is a copy)
 * correction = 1 - beta^step.
 * state_bits 32: m, v [n] fp32.  state_bits 8: m and r = sqrt(v) are kept in blocks
 * of 256 elements as e4m3 codes times a scale, the block's largest magnitude (at
 * least 1e-30) / 448; [n] codes, ceil(n / 256) scales.  The step itself uses m and
 * v before that rounding.  Rounding is stochastic: up with the chance of what
 * rounding down would leave, from 16 bits for each of m and r that follow from
 * `seed` and first + i (element i's number) alone:
 *   u = (first + i) * 0x9E3779B9 + ((first + i) >> 32) * 0x3C6EF373 + seed,
 *   u = (u ^ u >> 16) * 0x6A09E667,  u = (u ^ u >> 15) * 0xBB67AE85,  u ^= u >> 16
 * (32 bits), m's in the low half, r's in the high half; another seed for every
 * step.  An r > 0 is not rounded to 0.  A block with an infinity or NaN gets codes
 * 0 and a scale of NaN.
 * param, m, v, scales and copies are updated in place; they are 16-byte aligned, as
 * grad is, the scales 4, and no two of them may overlap.  n 0: left out. */
typedef struct {
  float *param;             /* [n]                                            */
  const void *grad;         /* [n] of grad_dtype                              */
  void *m, *v;              /* [n] fp32, or codes                             */
  float *mscale, *vscale;   /* [ceil(n / 256)] (state_bits 8)                 */
  void *copy;               /* [n] bf16, or NULL                              */
  long long n;              /* 0 <= n <= 2^39                                 */
  long long first;          /* number of element 0, >= 0 (state_bits 8)       */
  float decay;              /* weight decay                                   */
} twell_adamw_tensor;

/* What changes from step to step, in device memory (16-byte aligned), for a step
 * that is captured once and replayed: the caller writes it before each replay. */
typedef struct {
  float lr, correction1, correction2;
  uint32_t seed;
} twell_adamw_dynamic;

/* tensors: [count] in host memory, read before the call returns.  grad_scale: a
 * device scalar or NULL (1); where it is not finite, nothing is changed.  dynamic:
 * NULL, or in the place of lr, step and seed.  0 <= beta < 1, eps >= 0, 1 <= step,
 * all finite. */
twell_status twell_adamw_step(const twell_adamw_tensor *tensors, int count, int grad_dtype,
                              int state_bits, float lr, float beta1, float beta2, float eps,
                              long long step, uint32_t seed, const float *grad_scale,
                              const twell_adamw_dynamic *dynamic, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TWELL_LM_H */
