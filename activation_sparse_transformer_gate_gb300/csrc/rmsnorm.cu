// rmsnorm.cu -- residual addition + root-mean-square norm, with an output in
// the row's type or in 8 bits, and its backward.
//
// forward   s = x + r (stored),  rstd = (mean s^2 + eps)^(-1/2),  y = s rstd w
//           8 bits: scale = max|y| / 127,  q = rint(y / scale)
// backward  xhat = s rstd,  g = w dy
//           dx = ds + rstd (g - xhat mean(g xhat)),  dw = sum_t dy xhat
//
// HBM bounds both: every operand is read or written once.  A row stays in
// registers between the reduction and the output, spread over the fewest
// warps that keep at most NV 16-byte vectors a lane.  max|y| = rstd max|s w|,
// so the 8-bit output needs no second reduction.  16384 x 4096 bf16: forward
// 80 us (6.7 TB/s), with 8 bits out 78, backward 85 (6.3 TB/s; 81 right behind
// the forward, which leaves some of s in L2).
#include <float.h>

#include "common.cuh"
#include "lm_kernels.h"
#include "vec16.cuh"

namespace twell {

namespace {

constexpr int WARPS = 8;       // per CTA
constexpr int BWD_WARPS = 16;  // of the backward, one CTA an SM

// Sum and (bitwise) maximum over the W warps that share a row.  The maximum
// of |v| is taken on the bit patterns: their order is the values' order, and
// a NaN is above every number, so it is not lost.
template <int W>
__device__ __forceinline__ void reduce_row(float &sum, uint32_t &top, float (*s_sum)[WARPS],
                                           uint32_t (*s_top)[WARPS], int buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (W == 1) return;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    s_sum[buf][warp] = sum;
    s_top[buf][warp] = top;
  }
  __syncthreads();
  const int w0 = warp / W * W;
  sum = 0.f;
  top = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    sum += s_sum[buf][w0 + i];
    top = max(top, s_top[buf][w0 + i]);
  }
}

// The 8-bit scale of a row whose largest magnitude is `top`, and the factors
// (up, inv) with q = rint(v * up * inv): a row below 2^-60 is scaled up first
// so that 127 / top stays finite.  Rows that hold an infinity or NaN get
// scale NaN and q 0 (inv = 0, and fin = false).
struct Q8Scale {
  float scale, up, inv;
  bool fin;
};
__device__ __forceinline__ Q8Scale q8_scale(uint32_t top_bits) {
  Q8Scale r;
  const float top = __uint_as_float(top_bits);
  r.fin = top_bits < 0x7F800000u;
  r.up = top < 0x1p-60f ? 0x1p+64f : 1.f;
  r.scale = r.fin ? top / 127.f : __uint_as_float(0x7FC00000u);
  r.inv = r.fin && top > 0.f ? 127.f / (top * r.up) : 0.f;
  return r;
}
__device__ __forceinline__ uint32_t q8_of(float v, const Q8Scale &c) {
  if (!c.fin) return 0;
  const int q = __float2int_rn(v * c.up * c.inv);
  return (uint32_t)max(-127, min(127, q)) & 0xFFu;
}

template <typename E> struct Q8Word;  // one vector's 8-bit values
template <> struct Q8Word<float> { typedef uint32_t type; };
template <> struct Q8Word<bf16> { typedef uint2 type; };
__device__ __forceinline__ void q8_pack(const float (&f)[4], const Q8Scale &c, uint32_t &w) {
  w = q8_of(f[0], c) | q8_of(f[1], c) << 8 | q8_of(f[2], c) << 16 | q8_of(f[3], c) << 24;
}
__device__ __forceinline__ void q8_pack(const float (&f)[8], const Q8Scale &c, uint2 &w) {
  w.x = q8_of(f[0], c) | q8_of(f[1], c) << 8 | q8_of(f[2], c) << 16 | q8_of(f[3], c) << 24;
  w.y = q8_of(f[4], c) | q8_of(f[5], c) << 8 | q8_of(f[6], c) << 16 | q8_of(f[7], c) << 24;
}

// N fp32 weights of vector v.
template <int N>
__device__ __forceinline__ void load_w(const float *w, int v, float (&f)[N]) {
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    const float4 a = *(const float4 *)(w + (size_t)v * N + j);
    f[j] = a.x; f[j + 1] = a.y; f[j + 2] = a.z; f[j + 3] = a.w;
  }
}

// W warps a row, NV vectors a lane.
template <typename E, int W, int NV>
__global__ void __launch_bounds__(WARPS * 32)
rmsnorm_forward_kernel(const uint4 *x, const uint4 *res, const float *weight, int T, int nv,
                       float inv_d, float eps, uint4 *s_out, uint4 *y, int8_t *q, float *qscale,
                       float *rstd_out) {
  pdl_begin();
  constexpr int N = VEC16<E>;
  __shared__ float s_sum[1][WARPS];
  __shared__ uint32_t s_top[1][WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * (WARPS / W) + warp / W;
  const bool row_ok = t < T;
  const int v0 = (warp % W) * 32 + lane;
  const size_t base = (size_t)(row_ok ? t : 0) * nv;
  uint4 a[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = v0 + i * W * 32;
    const bool ok = row_ok && v < nv;
    a[i] = ok ? ld_once(x + base + v) : make_uint4(0, 0, 0, 0);
    b[i] = ok && res ? ld_once(res + base + v) : make_uint4(0, 0, 0, 0);
  }
  float sum = 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = v0 + i * W * 32;
    if (!row_ok || v >= nv) continue;
    if (res) {
      float f[N], g[N];
      unpack(a[i], f, (E *)nullptr);
      unpack(b[i], g, (E *)nullptr);
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] += g[j];
      a[i] = pack16(f, (E *)nullptr);  // the stored sum is what the norm reads
    }
    if (s_out) s_out[base + v] = a[i];
    float f[N];
    unpack(a[i], f, (E *)nullptr);
#pragma unroll
    for (int j = 0; j < N; ++j) sum += f[j] * f[j];
    if (q) {
      float w[N];
      load_w(weight, v, w);
#pragma unroll
      for (int j = 0; j < N; ++j) top = max(top, __float_as_uint(fabsf(f[j] * w[j])));
    }
  }
  reduce_row<W>(sum, top, s_sum, s_top, 0);
  if (!row_ok) return;
  // (below the normal range, which with eps 0 a row of zeros reaches, rstd is 0: y
  // and the backward's terms are then 0 and not 0 * inf)
  const float var = sum * inv_d + eps;
  const float rstd = var < FLT_MIN ? 0.f : rsqrtf(var);
  // (rstd is NaN, or 0 with an infinite sum, when s has a NaN or infinity:
  // 0 * inf then makes the row's largest magnitude NaN too)
  const Q8Scale sc = q8_scale(__float_as_uint(fabsf(__uint_as_float(top) * rstd)));
  if (v0 == 0) {
    if (rstd_out) rstd_out[t] = rstd;
    if (q) qscale[t] = sc.scale;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = v0 + i * W * 32;
    if (v >= nv) break;
    float f[N], w[N];
    unpack(a[i], f, (E *)nullptr);
    load_w(weight, v, w);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = f[j] * rstd * w[j];
    if (y) y[base + v] = pack16(f, (E *)nullptr);
    if (q) {
      typename Q8Word<E>::type word;
      q8_pack(f, sc, word);
      ((typename Q8Word<E>::type *)q)[base + v] = word;
    }
  }
}

// Backward.  The row groups (W warps each) of one CTA an SM walk the rows; each
// thread keeps its columns' weights and its part of dw in registers over all
// its rows, and the CTA's sum of the latter goes to the workspace at the end.
// BWD_STAGES rows of each thread's operands are on their way through shared
// memory at any time: 16 warps an SM, all that the registers leave room for, do
// not keep enough of HBM busy with loads to registers (16384 x 4096 bf16: 100
// us so).  A row group meets at a barrier of its own, so that the groups of a
// CTA drift apart and their reductions hide under each other's copies (4096 x 8192:
// 49.5 us; two CTAs of 8 warps an SM whose groups share the CTA's barrier 57).
constexpr int BWD_STAGES = 4, BWD_NV = 2;

constexpr int BWD_RING = BWD_STAGES * 3 * BWD_NV * BWD_WARPS * 32 * 16;  // bytes

// Sum over the W warps of a row group; the group's threads meet at a barrier
// of their own.
template <int W>
__device__ __forceinline__ float sum_group(float sum, float *s_sum) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (W == 1) return sum;
  const int warp = threadIdx.x >> 5, w0 = warp / W * W;
  if ((threadIdx.x & 31) == 0) s_sum[warp] = sum;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / W), "n"(W * 32) : "memory");
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) sum += s_sum[w0 + i];
  return sum;
}

template <typename E, int W>
__global__ void __launch_bounds__(BWD_WARPS * 32)
rmsnorm_backward_kernel(const uint4 *s_in, const float *weight, const float *rstd_in,
                        const uint4 *dy, const uint4 *ds, int T, int nv, float inv_d, uint4 *dx,
                        float *part) {
  pdl_begin();
  constexpr int N = VEC16<E>, NV = BWD_NV, THREADS = BWD_WARPS * 32, GROUPS = BWD_WARPS / W;
  extern __shared__ uint4 ring[];  // [stage][operand][NV][thread]
  __shared__ float s_sum[2][BWD_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = (int)blockIdx.x * GROUPS + warp / W;
  const int groups = (int)gridDim.x * GROUPS;
  const int v0 = (warp % W) * 32 + lane;
  float dw[NV][N], w[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (v0 + i * W * 32 < nv) load_w(weight, v0 + i * W * 32, w[i]);
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i][j] = 0.f;
  }
  auto slot = [&](int st, int op, int i) { return ring + ((st * 3 + op) * NV + i) * THREADS + threadIdx.x; };
  auto fetch = [&](long long t, int st) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = v0 + i * W * 32;
      if (t < T && v < nv) {
        const size_t o = (size_t)t * nv + v;
        copy16_async(slot(st, 0, i), s_in + o);
        copy16_async(slot(st, 1, i), dy + o);
        if (ds) copy16_async(slot(st, 2, i), ds + o);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int st = 0; st < BWD_STAGES; ++st) fetch(group + (long long)st * groups, st);
  float rstd_next = group < T ? rstd_in[group] : 0.f;
  int st = 0, r = 0;
  for (long long t = group; t < T; t += groups, ++r) {
    const float rstd = rstd_next;
    rstd_next = t + groups < T ? rstd_in[t + groups] : 0.f;
    asm volatile("cp.async.wait_group %0;" ::"n"(BWD_STAGES - 1) : "memory");
    uint4 a[NV], b[NV], c[NV];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (v0 + i * W * 32 >= nv) continue;
      a[i] = *slot(st, 0, i);
      b[i] = *slot(st, 1, i);
      c[i] = ds ? *slot(st, 2, i) : make_uint4(0, 0, 0, 0);
      float f[N], g[N];
      unpack(a[i], f, (E *)nullptr);
      unpack(b[i], g, (E *)nullptr);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float xhat = f[j] * rstd;
        dw[i][j] += g[j] * xhat;
        sum += g[j] * w[i][j] * xhat;
      }
    }
    fetch(t + (long long)BWD_STAGES * groups, st);
    st = st + 1 == BWD_STAGES ? 0 : st + 1;
    const float mean = sum_group<W>(sum, s_sum[r & 1]) * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = v0 + i * W * 32;
      if (v >= nv) continue;
      float f[N], g[N], h[N];
      unpack(a[i], f, (E *)nullptr);
      unpack(b[i], g, (E *)nullptr);
      unpack(c[i], h, (E *)nullptr);
#pragma unroll
      for (int j = 0; j < N; ++j) h[j] += rstd * (g[j] * w[i][j] - f[j] * rstd * mean);
      stg_stream(dx + (size_t)t * nv + v, pack16(h, (E *)nullptr));
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // the CTA's row groups in order, through the ring's memory
  float *sums = (float *)ring;  // [GROUPS][nv * N]
  const int D = nv * N;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = v0 + i * W * 32;
    if (v >= nv) break;
    float *p = sums + (size_t)(warp / W) * D + (size_t)v * N;
#pragma unroll
    for (int j = 0; j < N; j += 4)
      *(float4 *)(p + j) = make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
  }
  __syncthreads();
  for (int d = threadIdx.x * 4; d < D; d += THREADS * 4) {
    float4 acc = *(const float4 *)(sums + d);
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) {
      const float4 p = *(const float4 *)(sums + (size_t)i * D + d);
      acc.x += p.x; acc.y += p.y; acc.z += p.z; acc.w += p.w;
    }
    *(float4 *)(part + (size_t)blockIdx.x * D + d) = acc;
  }
}

// dw[d] = sum of the CTAs' rows of `part`: 32 columns a CTA, four a thread; 32
// threads take every 32nd row, and are added in order.
__global__ void __launch_bounds__(256)
rmsnorm_dw_kernel(const float *part, int rows, int D, float *dw) {
  pdl_begin();
  __shared__ float4 sums[32][8];
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int d = blockIdx.x * 32 + c * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (d < D)
#pragma unroll 10
    for (int r = g; r < rows; r += 32) {
      const float4 p = *(const float4 *)(part + (size_t)r * D + d);
      acc.x += p.x; acc.y += p.y; acc.z += p.z; acc.w += p.w;
    }
  sums[g][c] = acc;
  __syncthreads();
  if (g != 0 || d >= D) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) {
    const float4 p = sums[i][c];
    acc.x += p.x; acc.y += p.y; acc.z += p.z; acc.w += p.w;
  }
  dw[d] = acc.x; dw[d + 1] = acc.y; dw[d + 2] = acc.z; dw[d + 3] = acc.w;
}

// Symmetric 8-bit rows of a matrix: a CTA per row, which is read twice (the
// second time from L1 / L2).  For weights, once, so it is left plain: 14336 x 4096
// bf16 42 us (4.2 TB/s), 131072 x 4096 346 us (4.7 TB/s).
template <typename E>
__global__ void __launch_bounds__(256)
q8_quantize_kernel(const uint4 *a, int nv, int8_t *q, float *scale) {
  pdl_begin();
  constexpr int N = VEC16<E>;
  __shared__ float s_sum[1][WARPS];
  __shared__ uint32_t s_top[1][WARPS];
  const size_t base = (size_t)blockIdx.x * nv;
  uint32_t top = 0;
  for (int v = threadIdx.x; v < nv; v += 256) {
    float f[N];
    unpack(a[base + v], f, (E *)nullptr);
#pragma unroll
    for (int j = 0; j < N; ++j) top = max(top, __float_as_uint(fabsf(f[j])));
  }
  float none = 0.f;
  reduce_row<WARPS>(none, top, s_sum, s_top, 0);
  const Q8Scale sc = q8_scale(top);
  if (threadIdx.x == 0) scale[blockIdx.x] = sc.scale;
  for (int v = threadIdx.x; v < nv; v += 256) {
    float f[N];
    unpack(a[base + v], f, (E *)nullptr);
    typename Q8Word<E>::type word;
    q8_pack(f, sc, word);
    ((typename Q8Word<E>::type *)q)[base + v] = word;
  }
}

constexpr int FWD_NV = 2;  // vectors a lane before a row takes more warps

// The backward's CTAs: one an SM, fewer where their row groups cover the rows.
int backward_grid(int T, int nv) {
  int w = 1;  // warps of a row
  while (w < BWD_WARPS && nv > w * 32 * BWD_NV) w *= 2;
  const int per = BWD_WARPS / w;
  const int want = (T + per - 1) / per;
  return want < num_sms() ? want : num_sms();
}

template <typename E, int W, int NV>
cudaError_t forward_t(const void *x, const void *residual, const float *weight, int T, int nv,
                      float eps, void *s_out, void *y, int8_t *q, float *qscale, float *rstd,
                      cudaStream_t s) {
  const int per = WARPS / W;
  return launch_k(rmsnorm_forward_kernel<E, W, NV>, dim3((T + per - 1) / per), dim3(WARPS * 32), 0,
                  s, (const uint4 *)x, (const uint4 *)residual, weight, T, nv,
                  1.f / (float)(nv * VEC16<E>), eps, (uint4 *)s_out, (uint4 *)y, q, qscale, rstd);
}

template <typename E, int W>
cudaError_t backward_t(const void *s_in, const float *weight, const float *rstd, const void *dy,
                       const void *ds, int T, int nv, void *dx, float *dweight, float *part,
                       cudaStream_t s) {
  const int grid = backward_grid(T, nv);
  // (the ring holds the row groups' sums at the end too: BWD_WARPS / W rows of
  // at most W * 32 * BWD_NV vectors in fp32)
  static_assert(BWD_RING >= BWD_WARPS * 32 * BWD_NV * VEC16<E> * 4, "the sums fit");
  static const cudaError_t attr =
      cudaFuncSetAttribute(rmsnorm_backward_kernel<E, W>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, BWD_RING);
  if (attr != cudaSuccess) return attr;
  cudaError_t e = launch_k(rmsnorm_backward_kernel<E, W>, dim3(grid), dim3(BWD_WARPS * 32),
                           BWD_RING, s, (const uint4 *)s_in, weight, rstd, (const uint4 *)dy,
                           (const uint4 *)ds, T, nv, 1.f / (float)(nv * VEC16<E>), (uint4 *)dx,
                           part);
  if (e != cudaSuccess) return e;
  prof_mark(KID_RMSNORM_BWD, s);
  const int D = nv * VEC16<E>;
  e = launch_k(rmsnorm_dw_kernel, dim3((D + 31) / 32), dim3(256), 0, s, (const float *)part, grid,
               D, dweight);
  prof_mark(KID_RMSNORM_DW, s);
  return e;
}

template <typename E>
cudaError_t backward_rows(const void *s_in, const float *weight, const float *rstd, const void *dy,
                          const void *ds, int T, int D, void *dx, float *dweight, float *part,
                          cudaStream_t s) {
  const int nv = D / VEC16<E>;
  auto f = nv <= 64    ? backward_t<E, 1>
           : nv <= 128 ? backward_t<E, 2>
           : nv <= 256 ? backward_t<E, 4>
           : nv <= 512 ? backward_t<E, 8>
                       : backward_t<E, 16>;
  static_assert(BWD_NV == 2 && BWD_WARPS == 16, "rows of up to 1024 vectors");
  return f(s_in, weight, rstd, dy, ds, T, nv, dx, dweight, part, s);
}

// f<E, W, NV>(args...) for the row's width: at most FWD_NV vectors a lane up to
// eight warps, four beyond.
#define TWELL_ROW_DISPATCH(F, E, nv, most, ...)             \
  (nv <= 32 * most      ? F<E, 1, most>(__VA_ARGS__)        \
   : nv <= 64 * most    ? F<E, 2, most>(__VA_ARGS__)        \
   : nv <= 128 * most   ? F<E, 4, most>(__VA_ARGS__)        \
   : nv <= 256 * most   ? F<E, 8, most>(__VA_ARGS__)        \
                        : F<E, 8, 4>(__VA_ARGS__))

}  // namespace

cudaError_t launch_add_rmsnorm_forward(const void *x, const void *residual, const float *weight,
                                       int T, int D, int dtype, float eps, void *s_out, void *y,
                                       int8_t *q, float *qscale, float *rstd, cudaStream_t s) {
  cudaError_t e;
  if (dtype == TWELL_BF16) {
    const int nv = D / VEC16<bf16>;
    e = TWELL_ROW_DISPATCH(forward_t, bf16, nv, FWD_NV, x, residual, weight, T, nv, eps, s_out, y,
                           q, qscale, rstd, s);
  } else {
    const int nv = D / VEC16<float>;
    e = TWELL_ROW_DISPATCH(forward_t, float, nv, FWD_NV, x, residual, weight, T, nv, eps, s_out, y,
                           q, qscale, rstd, s);
  }
  prof_mark(KID_RMSNORM_FWD, s);
  return e;
}

size_t rmsnorm_scratch(int T, int D) {
  int grid = 0;  // of either type
  for (int n : {VEC16<bf16>, VEC16<float>}) {
    const int g = backward_grid(T, (D + n - 1) / n);
    if (g > grid) grid = g;
  }
  return (size_t)grid * (size_t)D * 4;
}

cudaError_t launch_add_rmsnorm_backward(const void *s_in, const float *weight, const float *rstd,
                                        const void *dy, const void *ds, int T, int D, int dtype,
                                        void *dx, float *dweight, float *part, cudaStream_t s) {
  return dtype == TWELL_BF16
             ? backward_rows<bf16>(s_in, weight, rstd, dy, ds, T, D, dx, dweight, part, s)
             : backward_rows<float>(s_in, weight, rstd, dy, ds, T, D, dx, dweight, part, s);
}

cudaError_t launch_q8_quantize(const void *a, int rows, int cols, int dtype, int8_t *q,
                               float *scale, cudaStream_t s) {
  cudaError_t e =
      dtype == TWELL_BF16
          ? launch_k(q8_quantize_kernel<bf16>, dim3(rows), dim3(256), 0, s, (const uint4 *)a,
                     cols / VEC16<bf16>, q, scale)
          : launch_k(q8_quantize_kernel<float>, dim3(rows), dim3(256), 0, s, (const uint4 *)a,
                     cols / VEC16<float>, q, scale);
  prof_mark(KID_Q8_QUANTIZE, s);
  return e;
}

}  // namespace twell
