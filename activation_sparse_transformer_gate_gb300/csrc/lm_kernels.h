// lm_kernels.h -- host-side launchers of the operators around the FFN
// (include/twell_lm.h; internal to libtwell).
#pragma once

#include "kernels.h"
#include "twell_lm.h"

namespace twell {

// embed.cu
struct EmbedArgs {
  const void *tokens;
  int token_bytes;          // 4 or 8
  int T, V, D, dtype;
  float scale;
  long long pad_id;
  int32_t *status;
};
// Scratch of the embedding gradient.
struct EmbedScratch {
  uint32_t *key[2];         // [T] sort keys (token, V for positions without one), ping-pong
  int32_t *pos[2];          // [T] their positions
  float *part;              // [chunks][2][D] sums of the runs that cross a chunk's ends
  size_t bytes;
};
EmbedScratch carve_embed(void *base, int T, int V, int D);
cudaError_t launch_embed_forward(const EmbedArgs &a, const void *table, void *out, cudaStream_t s);
cudaError_t launch_embed_backward(const EmbedArgs &a, const void *dy, float *dtable,
                                  const EmbedScratch &w, cudaStream_t s);

// rmsnorm.cu
cudaError_t launch_add_rmsnorm_forward(const void *x, const void *residual, const float *weight,
                                       int T, int D, int dtype, float eps, void *s_out, void *y,
                                       int8_t *q, float *qscale, float *rstd, cudaStream_t s);
size_t rmsnorm_scratch(int T, int D);
cudaError_t launch_add_rmsnorm_backward(const void *s_in, const float *weight, const float *rstd,
                                        const void *dy, const void *ds, int T, int D, int dtype,
                                        void *dx, float *dweight, float *part, cudaStream_t s);
cudaError_t launch_q8_quantize(const void *a, int rows, int cols, int dtype, int8_t *q,
                               float *scale, cudaStream_t s);

// distill.cu
constexpr int DISTILL_MAX_K = 256;  // entries of a teacher list
struct DistillArgs {
  const void *z;
  long long ldz;
  const int32_t *ids;
  const float *teacher;
  const float *row_weight;  // forward: NULL = all 1; backward: row_grad
  int T, V, k, dtype;
  float tau;
  float *loss, *stats;      // backward: loss NULL, stats read
  void *dz;
  int32_t *status;
};
cudaError_t launch_distill_forward(const DistillArgs &a, cudaStream_t s);
cudaError_t launch_distill_backward(const DistillArgs &a, cudaStream_t s);

// q8.cu
struct Q8Args {
  const int8_t *aq, *wq;
  const float *ascale, *wscale, *bias;
  int M, N, K, dtype;
  void *y;
  int32_t *status;
  void *ws;
};
constexpr int Q8_MAX_K = 65536;
size_t q8_scratch(int M, int N, int K);
cudaError_t launch_q8_matmul(const Q8Args &a, cudaStream_t s);

}  // namespace twell
