// recur.cu -- gated linear recurrence over packed sequences, and its backward.
//
//   a = sigmoid(gate + bias), c = 1 - a,  h_t = h_{t-1} + c_t (x_t - h_{t-1})
//   G_t = dh_t + a_{t+1} G_{t+1},  dx = c G,  dgate = G (h_{t-1} - x) a c
//
// A thread takes 16 bytes of channels through all rows.
#include "common.cuh"
#include "lm_kernels.h"
#include "vec16.cuh"

namespace twell {

namespace {

struct RecurParams {
  const int32_t *starts;
  int B, T, D;
  long long ld;
  const float *bias, *h0;
  float *hT, *states;
  const float *dhT;
  float *dbias, *dh0;
  int32_t *status;
};

// a = sigmoid(f) and c = 1 - a, each to a few units of its own last place.
__device__ __forceinline__ void gates(float f, float &a, float &c) {
  const float e = __expf(-fabsf(f)), big = __frcp_rn(1.f + e), small = e * big;
  a = f >= 0.f ? big : small;
  c = f >= 0.f ? small : big;
  if (f != f) a = c = f;
}

__device__ __forceinline__ void bounds(const RecurParams &p, int s, int &a, int &b) {
  a = p.starts ? p.starts[s] : (int)((long long)p.T / p.B * s);
  b = p.starts ? p.starts[s + 1] : (int)((long long)p.T / p.B * (s + 1));
  if (a < 0 || b > p.T || a > b) {
    set_status(p.status, TWELL_ERR_INDEX);
    b = a;
  }
}

template <typename E>
__global__ void recur_forward_kernel(const E *x, const E *gate, E *h, RecurParams p) {
  pdl_begin();
  constexpr int N = VEC16<E>;
  const int d = (blockIdx.x * blockDim.x + threadIdx.x) * N;
  if (d >= p.D) return;
  float b[N], y[N];
  for (int i = 0; i < N; ++i) b[i] = p.bias ? p.bias[d + i] : 0.f;
  for (int s = 0; s < p.B; ++s) {
    int ra, rb;
    bounds(p, s, ra, rb);
    for (int i = 0; i < N; ++i) y[i] = p.h0 ? p.h0[(size_t)s * p.D + d + i] : 0.f;
    for (int t = ra; t < rb; ++t) {
      float xv[N], gv[N];
      unpack(*(const uint4 *)(x + t * p.ld + d), xv, (E *)nullptr);
      unpack(*(const uint4 *)(gate + t * p.ld + d), gv, (E *)nullptr);
      if (p.states && t % RECUR_KEEP == 0)
        for (int i = 0; i < N; ++i) p.states[(size_t)(t / RECUR_KEEP) * p.D + d + i] = y[i];
      for (int i = 0; i < N; ++i) {
        float a, c;
        gates(gv[i] + b[i], a, c);
        y[i] = fmaf(c, xv[i] - y[i], y[i]);
      }
      *(uint4 *)(h + (size_t)t * p.D + d) = pack16(y, (E *)nullptr);
    }
    if (p.hT)
      for (int i = 0; i < N; ++i) p.hT[(size_t)s * p.D + d + i] = y[i];
  }
}

template <typename E>
__global__ void recur_backward_kernel(const E *x, const E *gate, const E *dh, E *dx, E *dgate,
                                      RecurParams p) {
  pdl_begin();
  constexpr int N = VEC16<E>;
  const int d = (blockIdx.x * blockDim.x + threadIdx.x) * N;
  if (d >= p.D) return;
  float b[N], u[N], db[N];
  for (int i = 0; i < N; ++i) {
    b[i] = p.bias ? p.bias[d + i] : 0.f;
    db[i] = 0.f;
  }
  for (int s = p.B - 1; s >= 0; --s) {
    int ra, rb;
    bounds(p, s, ra, rb);
    for (int i = 0; i < N; ++i) u[i] = p.dhT ? p.dhT[(size_t)s * p.D + d + i] : 0.f;
    for (int t = rb - 1; t >= ra; --t) {
      float xv[N], gv[N], dv[N], y[N];
      // the state before row t, from the last one kept
      const int k = t / RECUR_KEEP * RECUR_KEEP, from = max(k, ra);
      for (int i = 0; i < N; ++i)
        y[i] = from == ra ? (p.h0 ? p.h0[(size_t)s * p.D + d + i] : 0.f)
                          : p.states[(size_t)(k / RECUR_KEEP) * p.D + d + i];
      for (int r = from; r < t; ++r) {
        unpack(*(const uint4 *)(x + r * p.ld + d), xv, (E *)nullptr);
        unpack(*(const uint4 *)(gate + r * p.ld + d), gv, (E *)nullptr);
        for (int i = 0; i < N; ++i) {
          float a, c;
          gates(gv[i] + b[i], a, c);
          y[i] = fmaf(c, xv[i] - y[i], y[i]);
        }
      }
      unpack(*(const uint4 *)(x + t * p.ld + d), xv, (E *)nullptr);
      unpack(*(const uint4 *)(gate + t * p.ld + d), gv, (E *)nullptr);
      unpack(*(const uint4 *)(dh + (size_t)t * p.D + d), dv, (E *)nullptr);
      for (int i = 0; i < N; ++i) {
        float a, c;
        gates(gv[i] + b[i], a, c);
        const float G = dv[i] + u[i], dg = G * (y[i] - xv[i]) * (a * c);
        u[i] = fmaf(-c, G, G);
        dv[i] = c * G;
        gv[i] = dg;
        db[i] += dg;
      }
      *(uint4 *)(dx + t * p.ld + d) = pack16(dv, (E *)nullptr);
      *(uint4 *)(dgate + t * p.ld + d) = pack16(gv, (E *)nullptr);
    }
    if (p.dh0)
      for (int i = 0; i < N; ++i) p.dh0[(size_t)s * p.D + d + i] = u[i];
  }
  if (p.dbias)
    for (int i = 0; i < N; ++i) p.dbias[d + i] = db[i];
}

RecurParams params_of(const RecurArgs &a) {
  RecurParams p;
  p.starts = a.starts; p.B = a.B; p.T = a.T; p.D = a.D; p.ld = a.ld; p.bias = a.bias; p.h0 = a.h0;
  p.hT = a.hT; p.states = a.states; p.dhT = a.dhT; p.dbias = a.dbias; p.dh0 = a.dh0;
  p.status = a.status;
  return p;
}

template <typename E>
cudaError_t forward_t(const RecurArgs &a, cudaStream_t s) {
  const int n = a.D / VEC16<E>;
  return launch_k(recur_forward_kernel<E>, dim3((n + 63) / 64), dim3(64), 0, s, (const E *)a.x,
                  (const E *)a.gate, (E *)a.h, params_of(a));
}

template <typename E>
cudaError_t backward_t(const RecurArgs &a, cudaStream_t s) {
  const int n = a.D / VEC16<E>;
  return launch_k(recur_backward_kernel<E>, dim3((n + 63) / 64), dim3(64), 0, s, (const E *)a.x,
                  (const E *)a.gate, (const E *)a.dh, (E *)a.dx, (E *)a.dgate, params_of(a));
}

}  // namespace

cudaError_t launch_recur_forward(const RecurArgs &a, cudaStream_t s) {
  return a.dtype == TWELL_BF16 ? forward_t<bf16>(a, s) : forward_t<float>(a, s);
}

cudaError_t launch_recur_backward(const RecurArgs &a, cudaStream_t s) {
  return a.dtype == TWELL_BF16 ? backward_t<bf16>(a, s) : backward_t<float>(a, s);
}

}  // namespace twell
