// distill.cu -- distillation from a teacher's top logits: loss, gradient.
//
//   p = softmax(teacher / tau) over the row's entries, q = softmax(z / tau)
//   loss = w tau^2 sum_i p_i (log p_i - log q_{id_i}),  dz = w tau (q - p)
//
// The logits are the whole cost: 2 bytes in and 2 out per entry in bf16, and
// one exponential for the sum and one for the gradient.  The forward with
// the gradient reads each logit once: a thread-block cluster takes a row,
// every CTA keeps its slice in shared memory while it forms the running
// maximum and sum, the CTAs exchange those through distributed shared
// memory, and the slice is written out as the gradient.  The entries of the
// teacher's list are then patched by the CTA whose slice holds them, so p is
// never spread over the vocabulary.
//
// Exponentials are ex2((z - max z) * log2(e) / tau): the difference first, so
// that logits of the type's lowest value neither overflow nor, in a row of
// nothing else, lose the uniform q.
#include <cooperative_groups.h>

#include "common.cuh"
#include "lm_kernels.h"
#include "vec16.cuh"

namespace cg = cooperative_groups;

namespace twell {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int MAX_WARPS = 32;
constexpr int MAX_CLUSTER = 8;

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The reference that exponentials of a row (or part) with maximum m are taken
// against: m, or 0 where everything is -inf.
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

// (m, l) += (m2, l2): l counts exponentials against ref_of(m).
__device__ __forceinline__ void merge(float &m, float &l, float m2, float l2, float c) {
  const float top = fmaxf(m, m2);
  const float r = ref_of(top);
  l = l * ex2((m - r) * c) + l2 * ex2((m2 - r) * c);
  m = top;
}

// A row as aligned 16-byte vectors: vector j holds the elements
// j*N - lead .. j*N - lead + N - 1.  Only vectors wholly inside the row are
// read or written as vectors (the others are shared with the rows beside it).
template <typename E>
struct Row {
  const E *z;   // element 0
  int lead;     // elements between the aligned address below z and z
  int V, nvec;
  __device__ Row(const E *p, int V_) : z(p), V(V_) {
    lead = (int)(((uintptr_t)p & 15u) / sizeof(E));
    nvec = (int)(((long long)V + lead + VEC16<E> - 1) / VEC16<E>);
  }
  __device__ long long first(int j) const { return (long long)j * VEC16<E> - lead; }
  __device__ bool whole(int j) const { return first(j) >= 0 && first(j) + VEC16<E> <= V; }
};

template <typename E> __device__ __forceinline__ E lowest();
template <> __device__ __forceinline__ float lowest<float>() { return -INFINITY; }
template <> __device__ __forceinline__ bf16 lowest<bf16>() {
  return __ushort_as_bfloat16((unsigned short)0xFF80);
}

// Vector j of a row; elements outside it are -inf.
template <typename E>
__device__ __forceinline__ uint4 load_vec(const Row<E> &row, int j) {
  const long long e0 = row.first(j);
  if (row.whole(j)) return ld_once(row.z + e0);
  E e[VEC16<E>];
#pragma unroll
  for (int i = 0; i < VEC16<E>; ++i)
    e[i] = e0 + i >= 0 && e0 + i < row.V ? row.z[e0 + i] : lowest<E>();
  uint4 r;
  memcpy(&r, e, 16);
  return r;
}

template <typename E>
__device__ __forceinline__ void store_vec(const Row<E> &row, E *out, int j,
                                          const float (&f)[VEC16<E>]) {
  const long long e0 = row.first(j);
  if (row.whole(j)) {
    stg_stream(out + e0, pack16(f, (E *)nullptr));
    return;
  }
#pragma unroll
  for (int i = 0; i < VEC16<E>; ++i)
    if (e0 + i >= 0 && e0 + i < row.V) out[e0 + i] = from_f<E>(f[i]);
}

template <typename E>
__device__ __forceinline__ void store_zeros(const Row<E> &row, E *out, int j0, int j1) {
  float f[VEC16<E>];
#pragma unroll
  for (int i = 0; i < VEC16<E>; ++i) f[i] = 0.f;
  for (int j = j0 + (int)threadIdx.x; j < j1; j += blockDim.x) store_vec(row, out, j, f);
}

struct DistillParams {
  const int32_t *ids;
  const float *teacher;
  const float *w;
  long long ldz;
  int V, k;
  float tau, c, inv_tau;  // c = log2(e) / tau
  float *loss;
  float2 *stats;
  int32_t *status;
};

// The teacher's list of a row in shared memory.
struct Teacher {
  int id[DISTILL_MAX_K];     // -1: unused
  float t[DISTILL_MAX_K];    // teacher logit, then p
  float logp[DISTILL_MAX_K];
  float z[DISTILL_MAX_K];    // the student's logit there
};

// Thread i < k takes entry i; returns whether it is used.  An entry whose
// teacher logit is -inf has p = 0 and counts as unused.
template <typename E>
__device__ __forceinline__ bool load_entry(Teacher &te, const DistillParams &p, const E *z,
                                           size_t t) {
  const int i = threadIdx.x;
  if (i >= p.k) return false;
  int id = p.ids[t * p.k + i];
  const float v = p.teacher[t * p.k + i];
  if (id >= p.V) {
    set_status(p.status, TWELL_ERR_INDEX);
    id = -1;
  }
  if (v == -INFINITY) id = -1;
  te.id[i] = id < 0 ? -1 : id;
  te.t[i] = v;
  te.z[i] = id < 0 ? 0.f : to_f(z[id]);
  return id >= 0;
}

// p and log p of the list, by one warp (ends with a warp barrier).
__device__ __forceinline__ void teacher_softmax(Teacher &te, const DistillParams &p) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int i = lane; i < p.k; i += 32)
    if (te.id[i] >= 0) m = fmaxf(m, te.t[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float sum = 0.f;
  for (int i = lane; i < p.k; i += 32)
    if (te.id[i] >= 0) sum += ex2((te.t[i] - m) * p.c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  const float inv = 1.f / sum, ln = logf(sum);
  for (int i = lane; i < p.k; i += 32) {
    const bool on = te.id[i] >= 0;
    const float d = te.t[i] - m;
    te.t[i] = on ? ex2(d * p.c) * inv : 0.f;
    te.logp[i] = on ? d * p.inv_tau - ln : 0.f;
  }
  __syncwarp();
}

// Gradient at the list's entries that lie in vectors [j0, j1) of the row:
// entry i patches its element if it is the first with that id, with the
// probabilities of all of them.
template <typename E>
__device__ __forceinline__ void patch_entries(const Teacher &te, const DistillParams &p,
                                              const Row<E> &row, E *out, int j0, int j1, float ref,
                                              float nl, float g) {
  const int i = threadIdx.x;
  if (i >= p.k) return;
  const int id = te.id[i];
  const long long j = ((long long)id + row.lead) / VEC16<E>;
  if (id < 0 || j < j0 || j >= j1) return;
  float sum = 0.f;
  for (int o = 0; o < p.k; ++o) {
    if (te.id[o] != id) continue;
    if (o < i) return;
    sum += te.t[o];
  }
  out[id] = from_f<E>(g * (ex2((te.z[i] - ref) * p.c + nl) - sum));
}

// One cluster a row, CTA r of it the vectors [r * per, (r + 1) * per).  GRAD:
// the first `cap` of them stay in shared memory (all of them unless the row
// is longer than the cluster's shared memory; the rest is read again).
template <typename E, bool GRAD>
__global__ void __launch_bounds__(512)
distill_forward_kernel(const E *z, E *dz, DistillParams p, int cap) {
  pdl_begin();
  constexpr int N = VEC16<E>, U = 4;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const size_t t = blockIdx.x / C;
  const Row<E> row(z + t * p.ldz, p.V);
  E *out = GRAD ? dz + t * p.ldz : nullptr;
  const int per = (row.nvec + C - 1) / C;
  const int j0 = min(row.nvec, rank * per), j1 = min(row.nvec, j0 + per);
  const float w = p.w ? p.w[t] : 1.f;
  if (w == 0.f) {  // a masked row (uniform for the cluster): nothing is read
    if (GRAD) store_zeros(row, out, j0, j1);
    if (rank == 0 && threadIdx.x == 0) {
      p.loss[t] = 0.f;
      p.stats[t] = make_float2(0.f, 0.f);
    }
    return;
  }
  extern __shared__ uint4 slice[];
  __shared__ Teacher te;
  __shared__ float s_m[MAX_WARPS], s_l[MAX_WARPS];
  __shared__ float2 s_part;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool used = load_entry(te, p, row.z, t);

  float m = -INFINITY, l = 0.f;
  for (int j = j0 + (int)threadIdx.x; j < j1; j += U * blockDim.x) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j + u * (int)blockDim.x < j1) r[u] = load_vec(row, j + u * blockDim.x);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = j + u * (int)blockDim.x;
      if (at >= j1) break;
      if (GRAD && at - j0 < cap) slice[at - j0] = r[u];
      float f[N];
      unpack(r[u], f, (E *)nullptr);
      float top = f[0];
#pragma unroll
      for (int i = 1; i < N; ++i) top = fmaxf(top, f[i]);
      if (top > m) {
        l *= ex2((m - top) * p.c);
        m = top;
      }
      const float ref = ref_of(m);
#pragma unroll
      for (int i = 0; i < N; ++i) l += ex2((f[i] - ref) * p.c);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    merge(m, l, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, l, o), p.c);
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  const bool any = __syncthreads_or(used) != 0;
  if (warp == 0) {
    m = lane < (int)blockDim.x / 32 ? s_m[lane] : -INFINITY;
    l = lane < (int)blockDim.x / 32 ? s_l[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      merge(m, l, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, l, o), p.c);
    if (lane == 0) s_part = make_float2(m, l);
  } else if (warp == 1 && any) {
    teacher_softmax(te, p);
  }
  cluster.sync();
  m = -INFINITY;
  l = 0.f;
  for (int i = 0; i < C; ++i) {
    const float2 o = *cluster.map_shared_rank(&s_part, i);
    merge(m, l, o.x, o.y, p.c);
  }
  // (the CTAs' shared memory is read no more: the matching wait is at the end)
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  const float ref = ref_of(m);
  if (rank == 0 && warp == 0) {
    const float lnl = logf(l);
    float sum = 0.f;
    if (any)
      for (int i = lane; i < p.k; i += 32)
        if (te.id[i] >= 0 && te.t[i] != 0.f)
          sum += te.t[i] * (te.logp[i] - ((te.z[i] - ref) * p.inv_tau - lnl));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) {
      p.loss[t] = any ? w * p.tau * p.tau * sum : 0.f;
      p.stats[t] = make_float2(m, lnl);
    }
  }
  if (GRAD) {
    if (!any) {
      store_zeros(row, out, j0, j1);
    } else {
      const float g = w * p.tau, nl = -log2f(l);
      for (int j = j0 + (int)threadIdx.x; j < j1; j += blockDim.x) {
        const uint4 r = j - j0 < cap ? slice[j - j0] : load_vec(row, j);
        float f[N];
        unpack(r, f, (E *)nullptr);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = g * ex2((f[i] - ref) * p.c + nl);
        store_vec(row, out, j, f);
      }
      __syncthreads();  // the vectors are written before their entries are patched
      patch_entries(te, p, row, out, j0, j1, ref, nl, g);
    }
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// The gradient from the forward's statistics: a CTA per row and 2048 vectors.
constexpr int BWD_SLAB = 2048;

template <typename E>
__global__ void __launch_bounds__(256)
distill_backward_kernel(const E *z, E *dz, DistillParams p, int slabs) {
  pdl_begin();
  constexpr int N = VEC16<E>, U = 4;
  const size_t t = blockIdx.x / slabs;
  const Row<E> row(z + t * p.ldz, p.V);
  E *out = dz + t * p.ldz;
  const int j0 = (int)(blockIdx.x % slabs) * BWD_SLAB, j1 = min(row.nvec, j0 + BWD_SLAB);
  const float w = p.w[t];
  if (w == 0.f) {
    store_zeros(row, out, j0, j1);
    return;
  }
  __shared__ Teacher te;
  const bool used = load_entry(te, p, row.z, t);
  if (!__syncthreads_or(used)) {
    store_zeros(row, out, j0, j1);
    return;
  }
  const float2 st = p.stats[t];
  const float ref = ref_of(st.x), nl = -st.y * LOG2E, g = w * p.tau;
  for (int j = j0 + (int)threadIdx.x; j < j1; j += U * blockDim.x) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j + u * 256 < j1) r[u] = load_vec(row, j + u * 256);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u * 256 >= j1) break;
      float f[N];
      unpack(r[u], f, (E *)nullptr);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = g * ex2((f[i] - ref) * p.c + nl);
      store_vec(row, out, j + u * 256, f);
    }
  }
  if (threadIdx.x < 32) teacher_softmax(te, p);
  __syncthreads();
  patch_entries(te, p, row, out, j0, j1, ref, nl, g);
}

DistillParams params_of(const DistillArgs &a) {
  DistillParams p;
  p.ids = a.ids; p.teacher = a.teacher; p.w = a.row_weight; p.ldz = a.ldz; p.V = a.V; p.k = a.k;
  p.tau = a.tau; p.c = LOG2E / a.tau; p.inv_tau = 1.f / a.tau;
  p.loss = a.loss; p.stats = (float2 *)a.stats; p.status = a.status;
  return p;
}

// Slices of at most 108 KB let two CTAs share an SM, so that one loads while
// the other writes.
constexpr int SLICE_VECS = 108 * 1024 / 16, SLICE_MAX = 200 * 1024 / 16;

template <typename E, bool GRAD>
cudaError_t forward_t(const DistillArgs &a, cudaStream_t s) {
  const int nvec = (int)(((long long)a.V + 2 * VEC16<E> - 2) / VEC16<E>);  // (any alignment)
  int C = 1;
  if (GRAD)
    while (C < MAX_CLUSTER && (nvec + C - 1) / C > SLICE_VECS) C *= 2;
  // few rows: split them until every SM has two CTAs or a slice is 16 KB
  while (C < MAX_CLUSTER && (long long)a.T * C < 2 * num_sms() && nvec / C >= 1024) C *= 2;
  const int per = (nvec + C - 1) / C;
  const int cap = !GRAD ? 0 : per < SLICE_MAX ? per : SLICE_MAX;
  auto kern = distill_forward_kernel<E, GRAD>;
  static const cudaError_t attr =
      GRAD ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  SLICE_MAX * 16)
           : cudaSuccess;
  if (attr != cudaSuccess) return attr;
  if ((long long)a.T * C > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return launch_clusters(kern, dim3((unsigned)(a.T * C)), dim3(per <= 1024 ? 256 : 512),
                         (size_t)cap * 16, C, s, (const E *)a.z, (E *)a.dz, params_of(a), cap);
}

template <typename E>
cudaError_t backward_t(const DistillArgs &a, cudaStream_t s) {
  const int nvec = (int)(((long long)a.V + 2 * VEC16<E> - 2) / VEC16<E>);
  const int slabs = (nvec + BWD_SLAB - 1) / BWD_SLAB;
  if ((long long)a.T * slabs > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return launch_k(distill_backward_kernel<E>, dim3((unsigned)((long long)a.T * slabs)), dim3(256),
                  0, s, (const E *)a.z, (E *)a.dz, params_of(a), slabs);
}

}  // namespace

cudaError_t launch_distill_forward(const DistillArgs &a, cudaStream_t s) {
  if (a.dtype == TWELL_BF16) return a.dz ? forward_t<bf16, true>(a, s) : forward_t<bf16, false>(a, s);
  return a.dz ? forward_t<float, true>(a, s) : forward_t<float, false>(a, s);
}

cudaError_t launch_distill_backward(const DistillArgs &a, cudaStream_t s) {
  return a.dtype == TWELL_BF16 ? backward_t<bf16>(a, s) : backward_t<float>(a, s);
}

}  // namespace twell
