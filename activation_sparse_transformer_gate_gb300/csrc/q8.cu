// q8.cu -- product of 8-bit rows: y[m][n] = sa[m] sw[n] sum_k a[m][k] w[n][k].
#include "common.cuh"
#include "lm_kernels.h"
#include "vec16.cuh"

namespace twell {

namespace {

// 64 x 64 outputs a CTA, 64 bytes of K at a time through shared memory, 4 x 4
// outputs a thread, dp4a: the integer sum is exact (K <= 65536).
template <typename E>
__global__ void __launch_bounds__(256)
q8_tile_kernel(const int8_t *a, const int8_t *w, const float *sa, const float *sw,
               const float *bias, int M, int N, int K, E *y) {
  pdl_begin();
  __shared__ int ta[64][17], tw[64][17];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int r = threadIdx.x >> 2, c = threadIdx.x & 3;  // staging: row, 16-byte vector
  const int tm = threadIdx.x >> 4, tn = threadIdx.x & 15;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 64) {
    const bool kin = k0 + c * 16 < K;
    const uint4 va = kin && m0 + r < M ? *(const uint4 *)(a + (size_t)(m0 + r) * K + k0 + c * 16)
                                       : make_uint4(0, 0, 0, 0);
    const uint4 vw = kin && n0 + r < N ? *(const uint4 *)(w + (size_t)(n0 + r) * K + k0 + c * 16)
                                       : make_uint4(0, 0, 0, 0);
    __syncthreads();
    ta[r][c * 4] = va.x; ta[r][c * 4 + 1] = va.y; ta[r][c * 4 + 2] = va.z; ta[r][c * 4 + 3] = va.w;
    tw[r][c * 4] = vw.x; tw[r][c * 4 + 1] = vw.y; tw[r][c * 4 + 2] = vw.z; tw[r][c * 4 + 3] = vw.w;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      int x[4], v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = ta[tm + 16 * i][k];
        v[i] = tw[tn + 16 * i][k];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(x[i], v[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + tm + 16 * i, n = n0 + tn + 16 * j;
      if (m < M && n < N)
        y[(size_t)m * N + n] =
            from_f<E>((float)acc[i][j] * sa[m] * sw[n] + (bias ? bias[n] : 0.f));
    }
}

template <typename E>
cudaError_t matmul_t(const Q8Args &a, cudaStream_t s) {
  return launch_k(q8_tile_kernel<E>, dim3((a.N + 63) / 64, (a.M + 63) / 64), dim3(256), 0, s, a.aq,
                  a.wq, a.ascale, a.wscale, a.bias, a.M, a.N, a.K, (E *)a.y);
}

}  // namespace

size_t q8_scratch(int M, int N, int K) {
  (void)M; (void)N; (void)K;
  return 256;
}

cudaError_t launch_q8_matmul(const Q8Args &a, cudaStream_t s) {
  const cudaError_t e = a.dtype == TWELL_BF16 ? matmul_t<bf16>(a, s) : matmul_t<float>(a, s);
  prof_mark(KID_Q8_MATMUL, s);
  return e;
}

}  // namespace twell
