// lm_abi.cu -- C entry points of the operators around the FFN: argument
// checks and scratch carve-up (see include/twell_lm.h).
#include <math.h>

#include "common.cuh"
#include "lm_kernels.h"

using namespace twell;

namespace {

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

constexpr int MAX_ROWS = 1 << 30;  // tokens, rows, output columns: sums of two stay in int32

size_t elem_size(int dtype) { return dtype == TWELL_BF16 ? 2 : 4; }

twell_status check_dtype(int dtype) {
  return dtype == TWELL_F32 || dtype == TWELL_BF16 ? TWELL_OK : TWELL_ERR_DTYPE;
}

twell_status check_scratch(const void *ws, size_t bytes, size_t need) {
  if (need == 0) return TWELL_OK;
  if (!ws || ((uintptr_t)ws & 255u) != 0 || bytes < need) return TWELL_ERR_WORKSPACE;
  return TWELL_OK;
}

constexpr int EMBED_MAX_D = 65536, RECUR_MAX_D = 65536;

twell_status check_embed(const EmbedArgs &a) {
  twell_status st = check_dtype(a.dtype);
  if (st != TWELL_OK) return st;
  if (a.token_bytes != 4 && a.token_bytes != 8) return TWELL_ERR_DTYPE;
  if (a.T < 1 || a.T > MAX_ROWS || a.V < 1 || a.V == 0x7FFFFFFF || a.D < 1 ||
      a.D > EMBED_MAX_D || !a.tokens || !a.status)
    return TWELL_ERR_ARG;
  if ((size_t)a.D * elem_size(a.dtype) % 16 != 0) return TWELL_ERR_ALIGN;
  if (((uintptr_t)a.tokens & (uintptr_t)(a.token_bytes - 1)) != 0 || !aligned4(a.status))
    return TWELL_ERR_ALIGN;
  return TWELL_OK;
}

EmbedArgs embed_args(const void *tokens, int token_bytes, int T, int V, int D, int dtype,
                     float scale, long long pad_id, int32_t *status) {
  EmbedArgs a;
  a.tokens = tokens; a.token_bytes = token_bytes; a.T = T; a.V = V; a.D = D; a.dtype = dtype;
  a.scale = scale; a.pad_id = pad_id; a.status = status;
  return a;
}

// Row width of the norm: 16 bytes to 16 KB, whole 16-byte vectors.
twell_status check_rows(int T, int D, int dtype) {
  twell_status st = check_dtype(dtype);
  if (st != TWELL_OK) return st;
  if (T < 1 || T > MAX_ROWS || D < 1) return TWELL_ERR_ARG;
  const size_t bytes = (size_t)D * elem_size(dtype);
  if (bytes > 16384) return TWELL_ERR_ARG;
  return bytes % 16 == 0 ? TWELL_OK : TWELL_ERR_ALIGN;
}

}  // namespace

extern "C" {

twell_status twell_read_status(int32_t *status, void *stream) {
  if (!status) return TWELL_ERR_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  int32_t host = 0;
  cudaError_t e = cudaMemcpyAsync(&host, status, sizeof(int32_t), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(status, 0, sizeof(int32_t), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? (twell_status)host : TWELL_ERR_CUDA;
}

twell_status twell_embed_forward(const void *tokens, int token_bytes, const void *table, int T,
                                 int V, int D, int dtype, float scale, long long pad_id,
                                 void *out, int32_t *status, void *stream) {
  const EmbedArgs a = embed_args(tokens, token_bytes, T, V, D, dtype, scale, pad_id, status);
  const twell_status st = check_embed(a);
  if (st != TWELL_OK) return st;
  if (!table || !out) return TWELL_ERR_ARG;
  if (!aligned16(table) || !aligned16(out)) return TWELL_ERR_ALIGN;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  const cudaError_t e = launch_embed_forward(a, table, out, s);
  prof_mark(KID_EMBED_FWD, s);
  return cuda_status(e);
}

size_t twell_embed_workspace_size(int T, int V, int D) {
  if (T < 1 || T > MAX_ROWS || V < 1 || V == 0x7FFFFFFF || D < 1 || D > EMBED_MAX_D || D % 4 != 0) return 0;
  return carve_embed(nullptr, T, V, D).bytes;
}

twell_status twell_embed_backward(const void *tokens, int token_bytes, const void *dy, int T,
                                  int V, int D, int dtype, float scale, long long pad_id,
                                  float *dtable, int32_t *status, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  const EmbedArgs a = embed_args(tokens, token_bytes, T, V, D, dtype, scale, pad_id, status);
  twell_status st = check_embed(a);
  if (st != TWELL_OK) return st;
  if (!dy || !dtable) return TWELL_ERR_ARG;
  if (!aligned16(dy) || !aligned16(dtable)) return TWELL_ERR_ALIGN;
  st = check_scratch(workspace, workspace_bytes, carve_embed(nullptr, T, V, D).bytes);
  if (st != TWELL_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  return cuda_status(launch_embed_backward(a, dy, dtable, carve_embed(workspace, T, V, D), s));
}

twell_status twell_add_rmsnorm_forward(const void *x, const void *residual, const float *weight,
                                       int T, int D, int dtype, float eps, void *s, void *y,
                                       int8_t *q, float *qscale, float *rstd, void *stream) {
  const twell_status st = check_rows(T, D, dtype);
  if (st != TWELL_OK) return st;
  if (!x || !weight || !(eps >= 0.f) || (residual && !s) || (!y && !q) || (q && !qscale))
    return TWELL_ERR_ARG;
  if (q && D % 16 != 0) return TWELL_ERR_ALIGN;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(s) ||
      !aligned16(y) || !aligned16(q) || !aligned4(qscale) || !aligned4(rstd))
    return TWELL_ERR_ALIGN;
  cudaStream_t st_ = (cudaStream_t)stream;
  prof_mark(KID_START, st_);
  return cuda_status(launch_add_rmsnorm_forward(x, residual, weight, T, D, dtype, eps, s, y, q,
                                                qscale, rstd, st_));
}

size_t twell_add_rmsnorm_workspace_size(int T, int D) {
  if (T < 1 || T > MAX_ROWS || D < 4 || D > 8192 || D % 4 != 0) return 0;
  return rmsnorm_scratch(T, D);
}

twell_status twell_add_rmsnorm_backward(const void *s, const float *weight, const float *rstd,
                                        const void *dy, const void *ds, int T, int D, int dtype,
                                        void *dx, float *dweight, void *workspace,
                                        size_t workspace_bytes, void *stream) {
  twell_status st = check_rows(T, D, dtype);
  if (st != TWELL_OK) return st;
  if (!s || !weight || !rstd || !dy || !dx || !dweight) return TWELL_ERR_ARG;
  if (!aligned16(s) || !aligned16(weight) || !aligned4(rstd) || !aligned16(dy) || !aligned16(ds) ||
      !aligned16(dx) || !aligned4(dweight))
    return TWELL_ERR_ALIGN;
  st = check_scratch(workspace, workspace_bytes, rmsnorm_scratch(T, D));
  if (st != TWELL_OK) return st;
  cudaStream_t st_ = (cudaStream_t)stream;
  prof_mark(KID_START, st_);
  return cuda_status(launch_add_rmsnorm_backward(s, weight, rstd, dy, ds, T, D, dtype, dx, dweight,
                                                 (float *)workspace, st_));
}

twell_status twell_q8_quantize(const void *a, int rows, int cols, int dtype, int8_t *q,
                               float *scale, void *stream) {
  const twell_status st = check_dtype(dtype);
  if (st != TWELL_OK) return st;
  if (!a || !q || !scale || rows < 1 || rows > MAX_ROWS || cols < 1 || cols > MAX_ROWS)
    return TWELL_ERR_ARG;
  if (cols % 16 != 0 || !aligned16(a) || !aligned16(q) || !aligned4(scale)) return TWELL_ERR_ALIGN;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  return cuda_status(launch_q8_quantize(a, rows, cols, dtype, q, scale, s));
}

size_t twell_q8_workspace_size(int M, int N, int K) {
  if (M < 1 || M > MAX_ROWS || N < 1 || N > MAX_ROWS || K < 16 || K % 16 != 0 || K > Q8_MAX_K)
    return 0;
  return q8_scratch(M, N, K);
}

twell_status twell_q8_matmul(const int8_t *aq, const float *ascale, const int8_t *wq,
                             const float *wscale, const float *bias, int M, int N, int K,
                             int dtype, void *y, int32_t *status, void *workspace,
                             size_t workspace_bytes, void *stream) {
  twell_status st = check_dtype(dtype);
  if (st != TWELL_OK) return st;
  if (!aq || !ascale || !wq || !wscale || !y || !status || M < 1 || M > MAX_ROWS || N < 1 ||
      N > MAX_ROWS || K < 1 || K > Q8_MAX_K)
    return TWELL_ERR_ARG;
  if (K % 16 != 0 || !aligned16(aq) || !aligned16(wq) || !aligned16(y) || !aligned4(ascale) ||
      !aligned4(wscale) || !aligned4(bias) || !aligned4(status))
    return TWELL_ERR_ALIGN;
  st = check_scratch(workspace, workspace_bytes, q8_scratch(M, N, K));
  if (st != TWELL_OK) return st;
  Q8Args a;
  a.aq = aq; a.wq = wq; a.ascale = ascale; a.wscale = wscale; a.bias = bias;
  a.M = M; a.N = N; a.K = K; a.dtype = dtype; a.y = y; a.status = status; a.ws = workspace;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  return cuda_status(launch_q8_matmul(a, s));
}

static twell_status check_distill(const DistillArgs &a) {
  const twell_status st = check_dtype(a.dtype);
  if (st != TWELL_OK) return st;
  if (!a.z || !a.ids || !a.teacher || !a.stats || !a.status || a.T < 1 || a.T > MAX_ROWS ||
      a.V < 1 || a.V > MAX_ROWS || a.ldz < a.V || a.k < 1 || a.k > DISTILL_MAX_K || !(a.tau >= 1e-4f) || !(a.tau <= 1e4f))
    return TWELL_ERR_ARG;
  if (!aligned16(a.z) || !aligned16(a.dz) || !aligned4(a.ids) || !aligned4(a.teacher) ||
      !aligned4(a.row_weight) || !aligned4(a.loss) || ((uintptr_t)a.stats & 7u) != 0 ||
      !aligned4(a.status))
    return TWELL_ERR_ALIGN;
  return TWELL_OK;
}

static DistillArgs distill_args(const void *z, long long ldz, const int32_t *ids,
                                const float *teacher, const float *row_weight, int T, int V, int k,
                                int dtype, float tau, float *loss, float *stats, void *dz,
                                int32_t *status) {
  DistillArgs a;
  a.z = z; a.ldz = ldz; a.ids = ids; a.teacher = teacher; a.row_weight = row_weight;
  a.T = T; a.V = V; a.k = k; a.dtype = dtype; a.tau = tau;
  a.loss = loss; a.stats = stats; a.dz = dz; a.status = status;
  return a;
}

twell_status twell_distill_forward(const void *z, long long ldz, const int32_t *ids,
                                   const float *teacher, const float *row_weight, int T, int V,
                                   int k, int dtype, float tau, float *loss, float *stats,
                                   void *dz, int32_t *status, void *stream) {
  const DistillArgs a = distill_args(z, ldz, ids, teacher, row_weight, T, V, k, dtype, tau, loss,
                                     stats, dz, status);
  const twell_status st = check_distill(a);
  if (st != TWELL_OK) return st;
  if (!loss) return TWELL_ERR_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  const cudaError_t e = launch_distill_forward(a, s);
  prof_mark(KID_DISTILL_FWD, s);
  return cuda_status(e);
}

twell_status twell_distill_backward(const void *z, long long ldz, const int32_t *ids,
                                    const float *teacher, const float *stats,
                                    const float *row_grad, int T, int V, int k, int dtype,
                                    float tau, void *dz, int32_t *status, void *stream) {
  const DistillArgs a = distill_args(z, ldz, ids, teacher, row_grad, T, V, k, dtype, tau, nullptr,
                                     const_cast<float *>(stats), dz, status);
  const twell_status st = check_distill(a);
  if (st != TWELL_OK) return st;
  if (!row_grad || !dz) return TWELL_ERR_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  const cudaError_t e = launch_distill_backward(a, s);
  prof_mark(KID_DISTILL_BWD, s);
  return cuda_status(e);
}

static twell_status check_recur(const RecurArgs &a) {
  const twell_status st = check_dtype(a.dtype);
  if (st != TWELL_OK) return st;
  if (!a.x || !a.gate || !a.status || a.T < 1 || a.T > MAX_ROWS || a.B < 1 || a.B > MAX_ROWS ||
      a.D < 1 || a.D > RECUR_MAX_D || a.ld < a.D || a.ld > (1ll << 34))
    return TWELL_ERR_ARG;
  if (!a.starts && a.T % a.B != 0) return TWELL_ERR_ARG;
  const size_t es = elem_size(a.dtype);
  if ((size_t)a.D * es % 16 != 0 || (size_t)a.ld * es % 16 != 0) return TWELL_ERR_ALIGN;
  if (!aligned16(a.x) || !aligned16(a.gate) || !aligned16(a.bias) || !aligned4(a.starts) ||
      !aligned16(a.h0) || !aligned4(a.status) || !aligned16(a.h) || !aligned16(a.hT) ||
      !aligned16(a.states) || !aligned16(a.dh) || !aligned16(a.dhT) || !aligned16(a.dx) ||
      !aligned16(a.dgate) || !aligned16(a.dbias) || !aligned16(a.dh0))
    return TWELL_ERR_ALIGN;
  return TWELL_OK;
}

int twell_recur_states(int T) {
  return T < 1 || T > MAX_ROWS ? 0 : (T + RECUR_KEEP - 1) / RECUR_KEEP;
}

twell_status twell_recur_forward(const void *x, const void *gate, long long ld, const float *bias,
                                 const int32_t *starts, int B, const float *h0, int T, int D,
                                 int dtype, void *h, float *hT, float *states, int32_t *status,
                                 void *stream) {
  RecurArgs a = {};
  a.x = x; a.gate = gate; a.ld = ld; a.bias = bias; a.starts = starts; a.B = B; a.h0 = h0;
  a.T = T; a.D = D; a.dtype = dtype; a.h = h; a.hT = hT; a.states = states; a.status = status;
  const twell_status st = check_recur(a);
  if (st != TWELL_OK) return st;
  if (!h) return TWELL_ERR_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  const cudaError_t e = launch_recur_forward(a, s);
  prof_mark(KID_RECUR_FWD, s);
  return cuda_status(e);
}

twell_status twell_recur_backward(const void *x, const void *gate, long long ld,
                                  const float *bias, const int32_t *starts, int B,
                                  const float *h0, const float *states, const void *dh,
                                  const float *dhT, int T, int D, int dtype, void *dx,
                                  void *dgate, float *dbias, float *dh0, int32_t *status,
                                  void *stream) {
  RecurArgs a = {};
  a.x = x; a.gate = gate; a.ld = ld; a.bias = bias; a.starts = starts; a.B = B; a.h0 = h0;
  a.states = const_cast<float *>(states); a.dh = dh; a.dhT = dhT; a.T = T; a.D = D;
  a.dtype = dtype; a.dx = dx; a.dgate = dgate; a.dbias = dbias; a.dh0 = dh0; a.status = status;
  const twell_status st = check_recur(a);
  if (st != TWELL_OK) return st;
  if (!states || !dh || !dx || !dgate) return TWELL_ERR_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  const cudaError_t e = launch_recur_backward(a, s);
  prof_mark(KID_RECUR_BWD, s);
  return cuda_status(e);
}

static twell_status check_policy(const PolicyArgs &a) {
  const twell_status st = check_dtype(a.dtype);
  if (st != TWELL_OK) return st;
  if (a.token_bytes != 4 && a.token_bytes != 8) return TWELL_ERR_DTYPE;
  if (!a.z || !a.tokens || !a.logp || !a.stats || !a.status || a.T < 1 || a.T > MAX_ROWS ||
      a.V < 1 || a.V > MAX_ROWS || a.ldz < a.V || !(a.tau >= 1e-4f) || !(a.tau <= 1e4f) ||
      !(a.clip_low >= 0.f) || !(a.clip_low <= 1.f) || !(a.clip_high >= 0.f) ||
      !isfinite(a.clip_high) || !(a.beta >= 0.f) || !isfinite(a.beta))
    return TWELL_ERR_ARG;
  if (((uintptr_t)a.tokens & (uintptr_t)(a.token_bytes - 1)) != 0 || !aligned16(a.z) ||
      !aligned16(a.dz) || !aligned4(a.old_logp) || !aligned4(a.ref_logp) ||
      !aligned4(a.advantage) || !aligned4(a.row_weight) || !aligned4(a.loss) ||
      !aligned4(a.logp) || ((uintptr_t)a.stats & 7u) != 0 || !aligned4(a.status))
    return TWELL_ERR_ALIGN;
  return TWELL_OK;
}

twell_status twell_policy_forward(const void *z, long long ldz, const void *tokens,
                                  int token_bytes, const float *old_logp, const float *ref_logp,
                                  const float *advantage, const float *row_weight, int T, int V,
                                  int dtype, float tau, float clip_low, float clip_high,
                                  float beta, float *loss, float *logp, float *stats, void *dz,
                                  int32_t *status, void *stream) {
  const PolicyArgs a = {z, ldz, tokens, token_bytes, old_logp, ref_logp, advantage, row_weight, T,
                        V, dtype, tau, clip_low, clip_high, beta, loss, logp, stats, dz, status};
  const twell_status st = check_policy(a);
  if (st != TWELL_OK) return st;
  if (advantage ? !loss : loss || dz) return TWELL_ERR_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  const cudaError_t e = launch_policy_forward(a, s);
  prof_mark(KID_POLICY_FWD, s);
  return cuda_status(e);
}

twell_status twell_policy_backward(const void *z, long long ldz, const void *tokens,
                                   int token_bytes, const float *old_logp, const float *ref_logp,
                                   const float *advantage, const float *logp, const float *stats,
                                   const float *row_grad, int T, int V, int dtype, float tau,
                                   float clip_low, float clip_high, float beta, void *dz,
                                   int32_t *status, void *stream) {
  const PolicyArgs a = {z, ldz, tokens, token_bytes, old_logp, ref_logp, advantage, row_grad, T,
                        V, dtype, tau, clip_low, clip_high, beta, nullptr,
                        const_cast<float *>(logp), const_cast<float *>(stats), dz, status};
  const twell_status st = check_policy(a);
  if (st != TWELL_OK) return st;
  if (!row_grad || !advantage || !dz) return TWELL_ERR_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  const cudaError_t e = launch_policy_backward(a, s);
  prof_mark(KID_POLICY_BWD, s);
  return cuda_status(e);
}

twell_status twell_adamw_step(const twell_adamw_tensor *tensors, int count, int grad_dtype,
                              int state_bits, float lr, float beta1, float beta2, float eps,
                              long long step, uint32_t seed, const float *grad_scale,
                              const twell_adamw_dynamic *dynamic, void *stream) {
  twell_status st = check_dtype(grad_dtype);
  if (st != TWELL_OK) return st;
  if (state_bits != 8 && state_bits != 32) return TWELL_ERR_DTYPE;
  if (!tensors || count < 1 || !isfinite(lr) || !(beta1 >= 0.f) || !(beta1 < 1.f) ||
      !(beta2 >= 0.f) || !(beta2 < 1.f) || !(eps >= 0.f) || !isfinite(eps) || step < 1)
    return TWELL_ERR_ARG;
  if (!aligned4(grad_scale) || !aligned16(dynamic)) return TWELL_ERR_ALIGN;
  for (int i = 0; i < count; ++i) {
    const twell_adamw_tensor &t = tensors[i];
    if (t.n < 0 || t.n > (1ll << 39) || t.first < 0 || !isfinite(t.decay)) return TWELL_ERR_ARG;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && (!t.mscale || !t.vscale)))
      return TWELL_ERR_ARG;
    if (!aligned16(t.param) || !aligned16(t.grad) || !aligned16(t.m) || !aligned16(t.v) ||
        !aligned4(t.mscale) || !aligned4(t.vscale) || !aligned16(t.copy))
      return TWELL_ERR_ALIGN;
  }
  AdamwArgs a;
  a.tensors = tensors; a.count = count; a.grad_dtype = grad_dtype; a.state_bits = state_bits;
  a.lr = lr; a.beta1 = beta1; a.beta2 = beta2; a.eps = eps; a.seed = seed;
  a.correction1 = 1.0 - pow((double)beta1, (double)step);
  a.correction2 = 1.0 - pow((double)beta2, (double)step);
  a.grad_scale = grad_scale; a.dynamic = dynamic;
  cudaStream_t s = (cudaStream_t)stream;
  prof_mark(KID_START, s);
  const cudaError_t e = launch_adamw(a, s);
  prof_mark(KID_ADAMW, s);
  return cuda_status(e);
}

}  // extern "C"
