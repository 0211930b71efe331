// softmax_rows.cuh -- rows of logits streamed for a softmax: the exponentials'
// reference, a row as 16-byte vectors, running maximum and sum, and the
// gradient of a vector.  Shared by the losses over a vocabulary.
//
// Exponentials are 2^(z c - ref), c = log2(e) / tau, one fma before the ex2:
// ref is max z * c rounded, and as the same ref stands in the sum and in the
// gradient, its rounding cancels.  Where the maximum is so large that this
// rounding is no longer a fraction of a power of two, or z c would overflow (rows
// masked with a huge negative value and nothing else), the difference z - max z is
// taken first.
#pragma once

#include "common.cuh"
#include "vec16.cuh"

namespace twell {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The reference that the exponentials of a row (or part of one) with maximum
// m are taken against.
struct Ref {
  float m, mc;  // m (0 where everything is -inf), and max * c rounded
  bool wide;    // taken against m itself instead of mc
  __device__ __forceinline__ Ref(float max, float c) {
    m = max == -INFINITY ? 0.f : max;
    mc = __fmul_rn(max, c);  // (one rounding everywhere: not to be fused)
    // (below 2^24 the largest exponential is within 2^(1/2) of 1; from 2^32 on the
    // rounding of mc alone could take it out of fp32's range)
    wide = !(fabsf(mc) < 0x1p24f);
  }
  // log2 of an exponential against this reference
  __device__ __forceinline__ float operator()(float z, float c) const {
    return wide ? (z - m) * c : fmaf(z, c, -mc);
  }
};

// What a sum of exponentials against the reference of maximum `max` is
// multiplied by to count against `to`.
__device__ __forceinline__ float rescale(float max, const Ref &to, float c) {
  const Ref from(max, c);
  // (one of each kind may be neighbours: max c and its rounding are told apart)
  if (from.wide) return ex2(to.wide ? (max - to.m) * c : fmaf(max, c, -to.mc));
  return ex2(to.wide ? fmaf(-to.m, c, from.mc) : from.mc - to.mc);
}

// (m, l) += (m2, l2): l counts exponentials against the reference of m.
__device__ __forceinline__ void merge(float &m, float &l, float m2, float l2, float c) {
  const float top = fmaxf(m, m2);
  const Ref to(top, c);
  l = l * rescale(m, to, c) + l2 * rescale(m2, to, c);
  m = top;
}

// A row as aligned 16-byte vectors: vector j holds the elements
// j*N - lead .. j*N - lead + N - 1.  The vectors wholly inside the row,
// [w0, w1), are split among the CTAs; the elements before and behind them (at
// most N - 1 each) are its ends, single elements of the row's first CTA.
template <typename E>
struct Row {
  const uint4 *base;  // vector 0
  int lead;           // elements between the aligned address below the row and the row
  int V, w0, w1;
  int head, tail;     // ends: [0, head) and [tail, V)
  __device__ __forceinline__ Row(const E *p, int V_) : V(V_) {
    lead = (int)(((uintptr_t)p & 15u) / sizeof(E));
    base = (const uint4 *)(p - lead);
    w0 = lead ? 1 : 0;
    w1 = max(w0, (int)((V + (unsigned)lead) / VEC16<E>));
    head = min(V, lead ? VEC16<E> - lead : 0);
    tail = max(head, min(V, w1 * VEC16<E> - lead));
  }
  // end element i, or -1
  __device__ __forceinline__ int end(int i) const {
    return i < head ? i : i < head + V - tail ? tail + i - head : -1;
  }
  // whether the CTA of vectors [ja, jb) has element e
  __device__ __forceinline__ bool owns(int e, int ja, int jb, bool first) const {
    if (e < head || e >= tail) return first;
    const int j = (int)(((unsigned)e + lead) / VEC16<E>);
    return j >= ja && j < jb;
  }
};

// Zeros in a row of the gradient (its alignment is the logits'): vectors
// [ja, jb), and the ends for the row's first CTA; by the first `threads`.
template <typename E>
__device__ __forceinline__ void store_zeros(const Row<E> &row, E *out, int ja, int jb, bool first,
                                            int threads) {
  for (int j = ja + (int)threadIdx.x; j < jb; j += threads)
    stg_stream((uint4 *)(out - row.lead) + j, make_uint4(0, 0, 0, 0));
  const int e = row.end(threadIdx.x);
  if (first && e >= 0) out[e] = from_f<E>(0.f);
}

// Gradient of a vector: gl times its exponentials.
template <typename E>
__device__ __forceinline__ void grad_vec(const uint4 &r, const Ref &ref, float c, float gl,
                                         float (&f)[VEC16<E>]) {
  unpack(r, f, (E *)nullptr);
  if (!ref.wide) {
#pragma unroll
    for (int i = 0; i < VEC16<E>; ++i) f[i] = gl * ex2(fmaf(f[i], c, -ref.mc));
  } else {
#pragma unroll
    for (int i = 0; i < VEC16<E>; ++i) f[i] = gl * ex2(ref(f[i], c));
  }
}

__device__ __forceinline__ float max_of(const uint4 &r, float *) {
  return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
               fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
}
__device__ __forceinline__ float max_of(const uint4 &r, bf16 *) {
  const __nv_bfloat162 *p = (const __nv_bfloat162 *)&r;
  const __nv_bfloat162 m = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
  return fmaxf(__low2float(m), __high2float(m));
}

// Running maximum and sum of exponentials.
template <typename E>
struct Running {
  float m = -INFINITY, l = 0.f;
  Ref ref;
  float c;
  __device__ __forceinline__ explicit Running(float c_) : ref(-INFINITY, c_), c(c_) {}
  __device__ __forceinline__ void raise(float top) {
    if (top > m) {
      ref = Ref(top, c);
      l *= rescale(m, ref, c);
      m = top;
    }
  }
  // U vectors, of which the i with i * step < n count.  Their maximum first:
  // raising the reference costs as much as a vector, and some lane of a warp
  // would raise it at nearly every vector of a short slice.
  template <int U>
  __device__ __forceinline__ void add(const uint4 (&r)[U], int n, int step) {
    constexpr int N = VEC16<E>;
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u * step < n) top = fmaxf(top, max_of(r[u], (E *)nullptr));
    raise(top);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * step >= n) break;
      float f[N];
      unpack(r[u], f, (E *)nullptr);
      if (!ref.wide) {
#pragma unroll
        for (int i = 0; i < N; ++i) l += ex2(fmaf(f[i], c, -ref.mc));
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) l += ex2(ref(f[i], c));
      }
    }
  }
  __device__ __forceinline__ void add(float z) {
    raise(z);
    l += ex2(ref(z, c));
  }
};

// (m, l) of a warp's lanes, the same bits in each of them (additions over
// exchanged lanes commute).
__device__ __forceinline__ void merge_warp(float &m, float &l, float c) {
  float top = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  l *= rescale(m, Ref(top, c), c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  m = top;
}

// L2 policy of what is read again soon.
__device__ __forceinline__ uint64_t keep_policy() {
  uint64_t pol;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// A thread's own stream through shared memory: vectors first, first + step,
// ... below `end` of a row, RING of them in flight (registers would hold half
// as many), taken two at a time: f(two vectors, how many of them, index of the
// first).
constexpr int RING = 8;
template <typename F>
__device__ __forceinline__ void stream_vectors(const uint4 *base, int first, int end, int step,
                                               uint4 *ring, int threads, uint64_t policy, F f) {
  uint4 *mine = ring + threadIdx.x;
  const uint4 *src = base + first;
#pragma unroll
  for (int s = 0; s < RING; s += 2) {
#pragma unroll
    for (int i = s; i < s + 2; ++i)
      if (first + i * step < end) copy16_async(mine + i * threads, src + i * step, policy);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  for (int j = first; j < end; j += RING * step) {
    src += RING * step;
#pragma unroll
    for (int s = 0; s < RING; s += 2) {
      if (j + s * step >= end) break;
      asm volatile("cp.async.wait_group %0;" ::"n"(RING / 2 - 1) : "memory");
      const uint4 r[2] = {mine[s * threads], mine[(s + 1) * threads]};
      const int n = j + (s + 1) * step < end ? 2 : 1;
#pragma unroll
      for (int i = s; i < s + 2; ++i)
        if (j + (RING + i) * step < end)
          copy16_async(mine + i * threads, src + i * step, policy);
      asm volatile("cp.async.commit_group;" ::: "memory");
      f(r, n, j + s * step);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Adds a row's vectors [ja, jb), streamed by the first `threads` threads.
template <typename E>
__device__ __forceinline__ void sum_vectors(Running<E> &sum, const Row<E> &row, int ja, int jb,
                                            uint4 *ring, int threads, uint64_t policy) {
  stream_vectors(row.base, ja + (int)threadIdx.x, jb, threads, ring, threads, policy,
                 [&](const uint4 (&r)[2], int n, int) { sum.add(r, n, 1); });
}

// Writes the gradient at a row's vectors [ja, jb), in the same way.
template <typename E>
__device__ __forceinline__ void grad_vectors(const Row<E> &row, E *out, int ja, int jb, uint4 *ring,
                                             int threads, const Ref &ref, float c, float gl) {
  uint4 *dst = (uint4 *)(out - row.lead);
  stream_vectors(row.base, ja + (int)threadIdx.x, jb, threads, ring, threads,
                 gather_policy<L2_FIRST>(), [&](const uint4 (&r)[2], int n, int j) {
#pragma unroll
                   for (int i = 0; i < 2; ++i) {
                     if (i == n) break;
                     float f[VEC16<E>];
                     grad_vec<E>(r[i], ref, c, gl, f);
                     stg_stream(dst + j + i * threads, pack16(f, (E *)nullptr));
                   }
                 });
}

}  // namespace twell
