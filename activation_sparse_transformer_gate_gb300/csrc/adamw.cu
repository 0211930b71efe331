// adamw.cu -- one AdamW step over many tensors, states in 32 or 8 bits.
//
// Nothing but bytes: 30 a parameter with fp32 states and gradients and a bf16
// copy, 18 with states in 8 bits.  The tensors' addresses travel in the launch's
// parameters, so a step is one launch for up to MAX_TENSORS of them, captures as
// it is, and reads no list from memory.  A warp takes blocks of 256 elements; the
// block's largest magnitudes, which the 8-bit codes are scaled by, stay within it.
//
// The state's arithmetic is rounded operation by operation (no fused
// multiply-add), and the square root is IEEE's, so that the stochastic rounding to
// 8 bits falls the same way wherever the formula is evaluated in fp32.
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"
#include "lm_kernels.h"
#include "vec16.cuh"

namespace twell {

namespace {

constexpr int BLOCK = 256;              // elements that share a scale: 8 of each lane
constexpr int WARPS = 8;
constexpr int MAX_TENSORS = 380;        // of a launch: their table fills its parameters

struct Entry {
  float *p;
  const void *g;
  void *m, *v;
  float *ms, *vs;
  bf16 *copy;
  long long n, first;
  float decay;
};

template <int N>
struct Table {
  Entry e[N];
  uint32_t end[N];  // chunks of the tensors up to and including this one
  int count;
};

struct Scalars {
  float b1, o1, b2, o2, eps;
  float lr, step, isq;  // step = lr / correction1, isq = 1 / sqrt(correction2)
  uint32_t seed;
  const float *grad_scale;
  const twell_adamw_dynamic *dyn;
};

// 16 random bits for each of two roundings of element i.
__device__ __forceinline__ uint32_t noise_of(unsigned long long i, uint32_t seed) {
  uint32_t u = (uint32_t)i * 0x9E3779B9u + (uint32_t)(i >> 32) * 0x3C6EF373u + seed;
  u = (u ^ (u >> 16)) * 0x6A09E667u;
  u = (u ^ (u >> 15)) * 0xBB67AE85u;
  return u ^ (u >> 16);
}

// y in [0, 448] (a rounding above at most) as e4m3, rounded down after the noise
// (16 bits, in place) has been added below the three mantissa bits: up with the
// chance of what is cut off, to 2^-16.  Below 2^-6 the code's step is 2^-9, which is
// the mantissa's step from 2^-6 to 2^-5.
__device__ __forceinline__ uint32_t to_code(float y, uint32_t noise) {
  const bool small = y < 0x1p-6f;
  if (small) y = __fadd_rn(y, 0x1p-6f);
  return (__float_as_uint(y) + noise - (small ? 968u << 20 : 960u << 20)) >> 20;
}

// The larger magnitude; NaN if there is one.
__device__ __forceinline__ float top_of(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// Four codes as values.
__device__ __forceinline__ void from_codes(uint32_t w, float (&f)[4]) {
  const __half2 a = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3));
  const __half2 b = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3));
  const float2 x = __half22float2(a), y = __half22float2(b);
  f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
}

__device__ __forceinline__ void load4(const float *p, float (&f)[4]) {
  const uint4 r = ld_once(p);
  unpack(r, f, (float *)nullptr);
}
__device__ __forceinline__ void load4(const bf16 *p, float (&f)[4]) {
  const uint2 r = *(const uint2 *)p;
  f[0] = bf_lo(r.x); f[1] = bf_hi(r.x); f[2] = bf_lo(r.y); f[3] = bf_hi(r.y);
}

// The element's step: p, m and the new v; r = sqrt(v).
struct Step {
  float b1, o1, b2, o2, eps, step, isq, shrink, gs;  // shrink = lr decay
  __device__ __forceinline__ void operator()(float &p, float g, float &m, float &v, float &r) const {
    g = __fmul_rn(g, gs);
    m = __fadd_rn(__fmul_rn(m, b1), __fmul_rn(g, o1));
    v = __fadd_rn(__fmul_rn(v, b2), __fmul_rn(__fmul_rn(g, g), o2));
    r = __fsqrt_rn(v);
    p = fmaf(-step, __fdividef(m, fmaf(r, isq, eps)), fmaf(-shrink, p, p));
  }
};

template <typename G, int BITS, int N>
__global__ void __launch_bounds__(32 * WARPS, 4)
adamw_kernel(const __grid_constant__ Table<N> table, const Scalars sc) {
  pdl_begin();
  // the tensor of this CTA's chunk of WARPS blocks
  int lo = 0, hi = table.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (blockIdx.x < table.end[mid]) hi = mid;
    else lo = mid + 1;
  }
  const Entry &e = table.e[lo];
  const long long chunk = (long long)blockIdx.x - (lo ? table.end[lo - 1] : 0);
  const int lane = threadIdx.x & 31;
  const long long block = chunk * WARPS + (threadIdx.x >> 5), i0 = block * BLOCK;
  if (i0 >= e.n) return;
  Step st{sc.b1, sc.o1, sc.b2, sc.o2, sc.eps, sc.step, sc.isq, sc.lr * e.decay, 1.f};
  uint32_t seed = sc.seed;
  if (sc.dyn) {
    const twell_adamw_dynamic d = *sc.dyn;
    st.step = d.lr / d.correction1;
    st.isq = 1.f / sqrtf(d.correction2);
    st.shrink = d.lr * e.decay;
    seed = d.seed;
  }
  if (sc.grad_scale) {
    st.gs = *sc.grad_scale;
    if (!isfinite(st.gs)) return;
  }
  const int left = (int)min((long long)BLOCK, e.n - i0);
  const G *g = (const G *)e.g + i0;
  float *p = e.p + i0;
  float ms = 0.f, vs = 0.f;
  if (BITS == 8) {
    ms = e.ms[block];
    vs = e.vs[block];
  }
  float P[2][4], M[2][4], R[2][4];  // (R: v for fp32 states, sqrt(v) for 8 bits)
  float topm = 0.f, topr = 0.f;     // largest magnitudes
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = h * 128 + lane * 4;
    float gr[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) P[h][i] = M[h][i] = 0.f;
    if (at + 4 <= left) {
      load4(p + at, P[h]);
      load4(g + at, gr);
      if (BITS == 32) {
        load4((const float *)e.m + i0 + at, M[h]);
        load4((const float *)e.v + i0 + at, v);
      } else {
        from_codes(*(const uint32_t *)((const uint8_t *)e.m + i0 + at), M[h]);
        from_codes(*(const uint32_t *)((const uint8_t *)e.v + i0 + at), v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i < left) {
          P[h][i] = p[at + i];
          gr[i] = to_f(g[at + i]);
          if (BITS == 32) {
            M[h][i] = ((const float *)e.m)[i0 + at + i];
            v[i] = ((const float *)e.v)[i0 + at + i];
          } else {
            float f[4];
            from_codes(((const uint8_t *)e.m)[i0 + at + i], f);
            M[h][i] = f[0];
            from_codes(((const uint8_t *)e.v)[i0 + at + i], f);
            v[i] = f[0];
          }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BITS == 8) {
        M[h][i] = __fmul_rn(M[h][i], ms);
        v[i] = __fmul_rn(v[i], vs);
        v[i] = __fmul_rn(v[i], v[i]);
      }
      float r;
      st(P[h][i], gr[i], M[h][i], v[i], r);
      R[h][i] = BITS == 32 ? v[i] : r;
      if (BITS == 8) {  // (elements that the tensor does not have are 0)
        topm = top_of(topm, M[h][i]);
        topr = top_of(topr, r);
      }
    }
  }
  uint32_t cm[2] = {0, 0}, cr[2] = {0, 0};
  if (BITS == 8) {
    // (as bits, magnitudes are ordered, with NaN above infinity)
    const uint32_t bm = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(topm) & 0x7FFFFFFFu);
    const uint32_t br = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(topr) & 0x7FFFFFFFu);
    const bool okm = bm < 0x7F800000u, okr = br < 0x7F800000u;
    const float tm = fmaxf(__uint_as_float(bm), 1e-30f), tr = fmaxf(__uint_as_float(br), 1e-30f);
    const float im = __fdiv_rn(448.f, tm), ir = __fdiv_rn(448.f, tr);
    if (lane == 0) {
      e.ms[block] = okm ? __fmul_rn(tm, 1.f / 448.f) : NAN;
      e.vs[block] = okr ? __fmul_rn(tr, 1.f / 448.f) : NAN;
    }
    const unsigned long long first = (unsigned long long)(e.first + i0 + lane * 4);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u = noise_of(first + h * 128 + i, seed);
        const uint32_t a = to_code(__fmul_rn(fabsf(M[h][i]), im), u << 4 & 0xFFFF0u);
        const uint32_t b = to_code(__fmul_rn(R[h][i], ir), u >> 12 & 0xFFFF0u);
        // (r > 0 exactly where its bits are not 0)
        cr[h] |= max(b, min(__float_as_uint(R[h][i]), 1u)) << (8 * i);
        cm[h] |= (a | (__float_as_uint(M[h][i]) >> 24 & 0x80u)) << (8 * i);
      }
      if (!okm) cm[h] = 0;
      if (!okr) cr[h] = 0;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = h * 128 + lane * 4;
    if (at + 4 <= left) {
      stg_stream(p + at, pack16(P[h], (float *)nullptr));
      if (BITS == 32) {
        stg_stream((float *)e.m + i0 + at, pack16(M[h], (float *)nullptr));
        stg_stream((float *)e.v + i0 + at, pack16(R[h], (float *)nullptr));
      } else {
        *(uint32_t *)((uint8_t *)e.m + i0 + at) = cm[h];
        *(uint32_t *)((uint8_t *)e.v + i0 + at) = cr[h];
      }
      if (e.copy)
        *(uint2 *)(e.copy + i0 + at) =
            make_uint2(pack_bf2(P[h][0], P[h][1]), pack_bf2(P[h][2], P[h][3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i < left) {
          p[at + i] = P[h][i];
          if (BITS == 32) {
            ((float *)e.m)[i0 + at + i] = M[h][i];
            ((float *)e.v)[i0 + at + i] = R[h][i];
          } else {
            ((uint8_t *)e.m)[i0 + at + i] = (uint8_t)(cm[h] >> (8 * i));
            ((uint8_t *)e.v)[i0 + at + i] = (uint8_t)(cr[h] >> (8 * i));
          }
          if (e.copy) e.copy[i0 + at + i] = __float2bfloat16_rn(P[h][i]);
        }
    }
  }
}

template <typename G, int BITS, int N>
cudaError_t launch_table(const Table<N> &t, const Scalars &sc, cudaStream_t s) {
  return launch_k(adamw_kernel<G, BITS, N>, dim3(t.end[t.count - 1]), dim3(32 * WARPS), 0, s, t, sc);
}

template <int N>
cudaError_t launch_t(const AdamwArgs &a, const Scalars &sc, cudaStream_t s) {
  Table<N> t;
  t.count = 0;
  unsigned long long chunks = 0;
  auto flush = [&]() -> cudaError_t {
    if (t.count == 0) return cudaSuccess;
    const cudaError_t e =
        a.grad_dtype == TWELL_BF16
            ? a.state_bits == 8 ? launch_table<bf16, 8>(t, sc, s) : launch_table<bf16, 32>(t, sc, s)
        : a.state_bits == 8 ? launch_table<float, 8>(t, sc, s)
                            : launch_table<float, 32>(t, sc, s);
    t.count = 0;
    chunks = 0;
    return e;
  };
  for (int i = 0; i < a.count; ++i) {
    const twell_adamw_tensor &x = a.tensors[i];
    if (x.n == 0) continue;
    const unsigned long long more = ((unsigned long long)x.n + BLOCK * WARPS - 1) / (BLOCK * WARPS);
    if (t.count == N || chunks + more > 0x7FFFFFFFull) {
      const cudaError_t e = flush();
      if (e != cudaSuccess) return e;
    }
    chunks += more;
    t.e[t.count] = Entry{x.param, x.grad, x.m, x.v, x.mscale, x.vscale, (bf16 *)x.copy, x.n, x.first,
                         x.decay};
    t.end[t.count++] = (uint32_t)chunks;
  }
  return flush();
}

}  // namespace

cudaError_t launch_adamw(const AdamwArgs &a, cudaStream_t s) {
  Scalars sc;
  sc.b1 = a.beta1; sc.o1 = (float)(1.0 - (double)a.beta1);
  sc.b2 = a.beta2; sc.o2 = (float)(1.0 - (double)a.beta2);
  sc.eps = a.eps; sc.lr = a.lr;
  sc.step = (float)((double)a.lr / a.correction1);
  sc.isq = (float)(1.0 / sqrt(a.correction2));
  sc.seed = a.seed; sc.grad_scale = a.grad_scale; sc.dyn = a.dynamic;
  return a.count <= 16 ? launch_t<16>(a, sc, s) : launch_t<MAX_TENSORS>(a, sc, s);
}

}  // namespace twell
