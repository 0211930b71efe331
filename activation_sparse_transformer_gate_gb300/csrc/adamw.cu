// adamw.cu -- one AdamW step over many tensors, states in 32 or 8 bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p - lr decay p - lr / c1 m / (sqrt(v) / sqrt(c2) + eps)
//
// Bytes bound it: 30 a parameter with fp32 states and gradients and a bf16 copy, 18
// with states in 8 bits, where the instructions (106 an element before the copies
// ahead) come close: 0.41e9 parameters 1.34 ms of a floor of 1.10 by bytes, issue
// slots 82% busy; fp32 states at the floor (1.43e9 parameters 6.1 ms, 6.4 by the
// copy rate).  The tensors' addresses travel in the launch's parameters, so a step is
// one launch for up to MAX_TENSORS of them, captures as it is, and reads no list from
// memory.  A warp takes blocks of 256 elements; the block's largest magnitudes, which
// the 8-bit codes are scaled by, stay within it.
//
// 8 bits: e4m3 codes hold m and sqrt(v), whose range is half of v's in octaves.  A
// step moves an average by a fraction 1 - beta of the difference, 1e-3 and less for
// v, where half a code's distance is 2^-5 to 2^-4 of the value: rounded to nearest it
// would never move.  Rounded up with the chance of what is cut off, it moves as much
// in the mean.  The state's arithmetic is rounded operation by operation (no fused
// multiply-add), and the square root is IEEE's, so that this rounding falls the same
// way wherever the formula is evaluated in fp32.
#include <cuda_fp8.h>
#include <math.h>
#include <string.h>

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
  uint32_t end[N];  // blocks of the tensors up to and including this one
  int count;
};

struct Scalars {
  float b1, o1, b2, o2, eps;
  float lr, step, isq;  // step = lr / correction1, isq = 1 / sqrt(correction2)
  uint32_t seed;
  const float *grad_scale;
  const twell_adamw_dynamic *dyn;
};

// 16 random bits for each of two roundings of an element, from its number times K1
// (the high half of the number: times K3) plus the seed.
constexpr uint32_t NOISE_K1 = 0x9E3779B9u, NOISE_K3 = 0x3C6EF373u;
__device__ __forceinline__ uint32_t mix(uint32_t u) {
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

// A block of 8-bit states on its way through shared memory.
template <typename G>
struct Stage {
  float p[BLOCK];
  G g[BLOCK];
  uint8_t m[BLOCK], v[BLOCK];
  float scale[4];  // of m, of v
};
constexpr int CTAS8 = 4;  // an SM

// `bytes` (a multiple of 16) from global memory, by a warp.
template <int BYTES>
__device__ __forceinline__ void fetch_bytes(void *dst, const void *src) {
  const uint64_t once = gather_policy<L2_FIRST>();
#pragma unroll
  for (int k = (int)(threadIdx.x & 31) * 16; k < BYTES; k += 512)
    copy16_async((char *)dst + k, (const char *)src + k, once);
}
// The first n of a block's elements, and zeros.
template <typename T>
__device__ __forceinline__ void fetch_some(T *dst, const T *src, int n) {
  for (int k = threadIdx.x & 31; k < BLOCK; k += 32) {
    if (k < n) dst[k] = src[k];
    else memset(&dst[k], 0, sizeof(T));
  }
}

template <typename T>
__device__ __forceinline__ void read4(const T *p, float (&f)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float4 r = *(const float4 *)p;
    f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
  } else if constexpr (sizeof(T) == 2) {
    const uint2 r = *(const uint2 *)p;
    f[0] = bf_lo(r.x); f[1] = bf_hi(r.x); f[2] = bf_lo(r.y); f[3] = bf_hi(r.y);
  } else {
    from_codes(*(const uint32_t *)p, f);
  }
}

// A block's step from what a lane has of it (elements h * 128 + lane * 4 + i; v of 8
// bits: r, both not yet scaled), and its outputs.
template <int BITS>
__device__ __forceinline__ void update_block(const Entry &e, const Step &st, long long i0, uint32_t seed,
                                             float (&P)[2][4], const float (&Gr)[2][4],
                                             float (&M)[2][4], float (&R)[2][4], float ms, float vs) {
  const int lane = threadIdx.x & 31;
  float topm = 0.f, topr = 0.f;  // largest magnitudes
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = R[h][i], r;
      if (BITS == 8) {
        M[h][i] = __fmul_rn(M[h][i], ms);
        v = __fmul_rn(v, vs);
        v = __fmul_rn(v, v);
      }
      st(P[h][i], Gr[h][i], M[h][i], v, r);
      R[h][i] = BITS == 32 ? v : r;
      if (BITS == 8) {  // (elements that the tensor does not have are 0)
        topm = top_of(topm, M[h][i]);
        topr = top_of(topr, r);
      }
    }
  uint32_t cm[2] = {0, 0}, cr[2] = {0, 0};
  if (BITS == 8) {
    // (as bits, magnitudes are ordered, with NaN above infinity)
    const uint32_t bm = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(topm) & 0x7FFFFFFFu);
    const uint32_t br = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(topr) & 0x7FFFFFFFu);
    const bool okm = bm < 0x7F800000u, okr = br < 0x7F800000u;
    // (one division: m's in the even lanes, r's in the odd ones)
    const float top = fmaxf(__uint_as_float(lane & 1 ? br : bm), 1e-30f), inv = __fdiv_rn(448.f, top);
    const float im = __shfl_sync(0xFFFFFFFFu, inv, 0), ir = __shfl_sync(0xFFFFFFFFu, inv, 1);
    if (lane < 2)
      (lane ? e.vs : e.ms)[i0 / BLOCK] = (lane ? okr : okm) ? __fmul_rn(top, 1.f / 448.f) : NAN;
    const unsigned long long first = (unsigned long long)(e.first + i0 + lane * 4);
    const uint32_t low = (uint32_t)first;
    const uint32_t u0 = low * NOISE_K1 + (uint32_t)(first >> 32) * NOISE_K3 + seed;
    const bool wraps = low > 0xFFFFFF00u;  // (the number's high half grows among these elements)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = h * 128 + i;
        uint32_t u = u0 + at * NOISE_K1;
        if (wraps && low + at < low) u += NOISE_K3;
        u = mix(u);
        const uint32_t a = to_code(__fmul_rn(fabsf(M[h][i]), im), u << 4 & 0xFFFF0u);
        const uint32_t c = to_code(__fmul_rn(R[h][i], ir), u >> 12 & 0xFFFF0u);
        // (r > 0 exactly where its bits are not 0)
        cr[h] |= max(c, min(__float_as_uint(R[h][i]), 1u)) << (8 * i);
        cm[h] |= (a | (__float_as_uint(M[h][i]) >> 24 & 0x80u)) << (8 * i);
      }
      if (!okm) cm[h] = 0;
      if (!okr) cr[h] = 0;
    }
  }
  if (i0 + BLOCK <= e.n) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long at = i0 + h * 128 + lane * 4;
      stg_stream(e.p + at, pack16(P[h], (float *)nullptr));
      if (BITS == 32) {
        stg_stream((float *)e.m + at, pack16(M[h], (float *)nullptr));
        stg_stream((float *)e.v + at, pack16(R[h], (float *)nullptr));
      } else {
        *(uint32_t *)((uint8_t *)e.m + at) = cm[h];
        *(uint32_t *)((uint8_t *)e.v + at) = cr[h];
      }
      if (e.copy)
        *(uint2 *)(e.copy + at) =
            make_uint2(pack_bf2(P[h][0], P[h][1]), pack_bf2(P[h][2], P[h][3]));
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long at = i0 + h * 128 + lane * 4 + i;
        if (at >= e.n) continue;
        e.p[at] = P[h][i];
        if (BITS == 32) {
          ((float *)e.m)[at] = M[h][i];
          ((float *)e.v)[at] = R[h][i];
        } else {
          ((uint8_t *)e.m)[at] = (uint8_t)(cm[h] >> (8 * i));
          ((uint8_t *)e.v)[at] = (uint8_t)(cr[h] >> (8 * i));
        }
        if (e.copy) e.copy[at] = __float2bfloat16_rn(P[h][i]);
      }
  }
}

// What a launch's scalars give (false: a step that is given up).
__device__ __forceinline__ bool open_step(const Scalars &sc, Step &st, float &lr, uint32_t &seed) {
  lr = sc.lr;
  seed = sc.seed;
  st = Step{sc.b1, sc.o1, sc.b2, sc.o2, sc.eps, sc.step, sc.isq, 0.f, 1.f};
  if (sc.dyn) {
    const twell_adamw_dynamic d = *sc.dyn;
    lr = d.lr;
    st.step = d.lr / d.correction1;
    st.isq = 1.f / sqrtf(d.correction2);
    seed = d.seed;
  }
  if (!sc.grad_scale) return true;
  st.gs = *sc.grad_scale;
  return isfinite(st.gs);
}

// Elements at .. at + 3 of n (zeros from n on), read once.
__device__ __forceinline__ void load_some(const float *p, long long at, long long n, float (&f)[4]) {
  if (at + 4 <= n) {
    unpack(ld_once(p + at), f, (float *)nullptr);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = at + i < n ? p[at + i] : 0.f;
  }
}
__device__ __forceinline__ void load_some(const bf16 *p, long long at, long long n, float (&f)[4]) {
  if (at + 4 <= n) {
    read4(p + at, f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = at + i < n ? __bfloat162float(p[at + i]) : 0.f;
  }
}

__device__ __forceinline__ void load_some(const uint8_t *p, long long at, long long n, float (&f)[4]) {
  uint32_t w = 0;
  if (at + 4 <= n) {
    w = *(const uint32_t *)(p + at);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i < n) w |= (uint32_t)p[at + i] << (8 * i);
  }
  from_codes(w, f);
}

// A warp a block, straight from global memory.
template <typename G, int BITS, int N>
__global__ void __launch_bounds__(32 * WARPS, 4)
adamw_direct_kernel(const __grid_constant__ Table<N> table, const Scalars sc) {
  pdl_begin();
  const long long b = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
  int lo = 0, hi = table.count - 1;
  if (b >= table.end[hi]) return;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (b < table.end[mid]) hi = mid;
    else lo = mid + 1;
  }
  const Entry &e = table.e[lo];
  const long long i0 = (b - (lo ? table.end[lo - 1] : 0)) * BLOCK;
  Step st;
  float lr;
  uint32_t seed;
  if (!open_step(sc, st, lr, seed)) return;
  st.shrink = lr * e.decay;
  float P[2][4], Gr[2][4], M[2][4], R[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long at = i0 + h * 128 + (threadIdx.x & 31) * 4;
    load_some(e.p, at, e.n, P[h]);
    load_some((const G *)e.g, at, e.n, Gr[h]);
    if (BITS == 32) {
      load_some((const float *)e.m, at, e.n, M[h]);
      load_some((const float *)e.v, at, e.n, R[h]);
    } else {
      load_some((const uint8_t *)e.m, at, e.n, M[h]);
      load_some((const uint8_t *)e.v, at, e.n, R[h]);
    }
  }
  const float ms = BITS == 8 ? e.ms[i0 / BLOCK] : 0.f, vs = BITS == 8 ? e.vs[i0 / BLOCK] : 0.f;
  update_block<BITS>(e, st, i0, seed, P, Gr, M, R, ms, vs);
}

// States in 8 bits: warps go over the blocks in strides of the grid, two of them on
// their way to shared memory while one is worked on (registers would hold one; a warp
// a block took 1577 us where this takes 1340).
template <typename G, int N>
__global__ void __launch_bounds__(32 * WARPS, CTAS8)
adamw8_kernel(const __grid_constant__ Table<N> table, const Scalars sc) {
  pdl_begin();
  using S = Stage<G>;
  extern __shared__ __align__(16) char shared[];
  S *const stages = (S *)shared + 2 * (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long blocks = table.end[table.count - 1], stride = (long long)gridDim.x * WARPS;
  Step st;
  float lr;
  uint32_t seed;
  if (!open_step(sc, st, lr, seed)) return;
  // the tensor of block b (b grows from call to call)
  auto advance = [&](int &t, long long b) {
    while (t < table.count - 1 && b >= table.end[t]) ++t;
  };
  auto fetch = [&](int t, long long b, S &sg) {
    const Entry &e = table.e[t];
    const long long block = b - (t ? table.end[t - 1] : 0), i0 = block * BLOCK;
    if (i0 + BLOCK <= e.n) {
      fetch_bytes<BLOCK * 4>(sg.p, e.p + i0);
      fetch_bytes<BLOCK * sizeof(G)>(sg.g, (const G *)e.g + i0);
      const bool second = lane >= 16;  // (the codes: 16 lanes each)
      copy16_async((second ? sg.v : sg.m) + (lane & 15) * 16,
                   (const char *)(second ? e.v : e.m) + i0 + (lane & 15) * 16,
                   gather_policy<L2_FIRST>());
    } else {
      const int n = (int)(e.n - i0);
      fetch_some(sg.p, (const float *)e.p + i0, n);
      fetch_some(sg.g, (const G *)e.g + i0, n);
      fetch_some(sg.m, (const uint8_t *)e.m + i0, n);
      fetch_some(sg.v, (const uint8_t *)e.v + i0, n);
    }
    if (lane < 2)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(&sg.scale[lane])),
                   "l"((lane ? e.vs : e.ms) + block)
                   : "memory");
  };
  long long b = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
  int t = 0, ahead = 0;  // tensors of the block worked on, and of the one fetched
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (b + k * stride < blocks) {
      advance(ahead, b + k * stride);
      fetch(ahead, b + k * stride, stages[k]);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  for (int k = 0; b < blocks; b += stride, k ^= 1) {
    S &sg = stages[k];
    advance(t, b);
    const Entry &e = table.e[t];
    const long long block = b - (t ? table.end[t - 1] : 0), i0 = block * BLOCK;
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    float P[2][4], Gr[2][4], M[2][4], R[2][4];  // (R: v for fp32 states, sqrt(v) for 8 bits)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = h * 128 + lane * 4;
      read4(sg.p + at, P[h]);
      read4(sg.g + at, Gr[h]);
      read4(sg.m + at, M[h]);
      read4(sg.v + at, R[h]);
    }
    const float ms = sg.scale[0], vs = sg.scale[1];
    __syncwarp();  // (all have read the stage)
    if (b + 2 * stride < blocks) {
      advance(ahead, b + 2 * stride);
      fetch(ahead, b + 2 * stride, sg);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    st.shrink = lr * e.decay;
    update_block<8>(e, st, i0, seed, P, Gr, M, R, ms, vs);
  }
}

template <typename G, int BITS, int N>
cudaError_t launch_direct(const Table<N> &t, const Scalars &sc, cudaStream_t s) {
  const long long ctas = (t.end[t.count - 1] + (long long)WARPS - 1) / WARPS;
  return launch_k(adamw_direct_kernel<G, BITS, N>, dim3((unsigned)ctas), dim3(32 * WARPS), 0, s, t, sc);
}

template <typename G, int N>
cudaError_t launch8(const Table<N> &t, const Scalars &sc, cudaStream_t s) {
  auto kern = adamw8_kernel<G, N>;
  constexpr int SMEM = 2 * WARPS * sizeof(Stage<G>);
  static const cudaError_t attr =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (attr != cudaSuccess) return attr;
  const long long ctas = (t.end[t.count - 1] + (long long)WARPS - 1) / WARPS;
  const long long most = (long long)num_sms() * CTAS8;
  // Fetching ahead pays from about two blocks a warp (us, ahead | direct: 0.53e6
  // parameters 5.4 | 3.9, 2.1e6 10.6 | 9.8, 5.1e6 21.6 | 24.9, 16.7e6 61 | 76, 255e6 824 | 1028).
  if (ctas <= 2 * most) return launch_direct<G, 8>(t, sc, s);
  return launch_k(kern, dim3((unsigned)(ctas < most ? ctas : most)), dim3(32 * WARPS), SMEM, s, t, sc);
}

template <int N>
cudaError_t launch_t(const AdamwArgs &a, const Scalars &sc, cudaStream_t s) {
  Table<N> t;
  t.count = 0;
  unsigned long long blocks = 0;
  auto flush = [&]() -> cudaError_t {
    if (t.count == 0) return cudaSuccess;
    const cudaError_t e =
        a.grad_dtype == TWELL_BF16
            ? a.state_bits == 8 ? launch8<bf16>(t, sc, s) : launch_direct<bf16, 32>(t, sc, s)
        : a.state_bits == 8 ? launch8<float>(t, sc, s)
                            : launch_direct<float, 32>(t, sc, s);
    t.count = 0;
    blocks = 0;
    return e;
  };
  for (int i = 0; i < a.count; ++i) {
    const twell_adamw_tensor &x = a.tensors[i];
    if (x.n == 0) continue;
    const unsigned long long more = ((unsigned long long)x.n + BLOCK - 1) / BLOCK;
    if (t.count == N || blocks + more > 0xFFFFFFFFull) {
      const cudaError_t e = flush();
      if (e != cudaSuccess) return e;
    }
    blocks += more;
    t.e[t.count] = Entry{x.param, x.grad, x.m, x.v, x.mscale, x.vscale, (bf16 *)x.copy, x.n, x.first,
                         x.decay};
    t.end[t.count++] = (uint32_t)blocks;
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
