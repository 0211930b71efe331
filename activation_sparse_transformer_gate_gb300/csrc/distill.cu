// distill.cu -- distillation from a teacher's top logits: loss, gradient.
//
//   p = softmax(teacher / tau) over the row's entries, q = softmax(z / tau)
//   loss = w tau^2 sum_i p_i (log p_i - log q_{id_i}),  dz = w tau (q - p)
//
// The logits are the whole cost: 2 bytes in and 2 out per entry in bf16, and
// one exponential for the sum and one for the gradient.  HBM bounds it, then
// the exponentials (16 a clock an SM).  The forward with the gradient reads
// each logit from HBM once; by the shape, a row belongs to
//   a warp            up to 256 vectors of 16 bytes
//   a CTA             many rows: it streams the row twice, the second time
//                     from L2
//   a cluster of CTAs few rows: each keeps its slice in shared memory, and
//                     maxima and sums go through distributed shared memory
// p is never spread over the vocabulary: the list's entries of the gradient
// are written over what the stream left there.
//
// One warp of each CTA deals with the teacher's list while the others stream
// the logits: its softmax, repeated ids, the student's logits there, the loss,
// and at the end the list's entries of the gradient.
#include <cooperative_groups.h>

#include "common.cuh"
#include "lm_kernels.h"
#include "softmax_rows.cuh"

namespace cg = cooperative_groups;

namespace twell {

namespace {

constexpr int MAX_WARPS = 7;     // streaming warps of a CTA (8 with the list's)
constexpr int MAX_CLUSTER = 8;

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

// The teacher's list of a row in shared memory, kept by one warp.
struct Teacher {
  int4 id4[DISTILL_MAX_K / 4];  // ids; -1: unused
  float p[DISTILL_MAX_K];       // teacher logit, then probability
  float logp[DISTILL_MAX_K];
  float z[DISTILL_MAX_K];       // the student's logit there
  float sum[DISTILL_MAX_K];     // of the probabilities with this id; -1: not the id's first entry
  int4 seen4[DISTILL_MAX_K / 2];  // hash table of the ids (twice their number, -1: free)
  __device__ __forceinline__ int *id() { return (int *)id4; }
};

// The list and the student's logits there, by one warp; z: the row.  Entries
// whose teacher logit is -inf have p = 0 and count as unused.  Returns whether
// any entry is used.
template <typename E>
__device__ __forceinline__ bool load_list(Teacher &te, const DistillParams &p, const E *z,
                                          size_t t) {
  const int lane = threadIdx.x & 31;
  bool any = false;
  for (int i = lane; i < (p.k + 3) / 4 * 4; i += 32) {
    int id = i < p.k ? p.ids[t * p.k + i] : -1;
    const float v = i < p.k ? p.teacher[t * p.k + i] : 0.f;
    if (id >= p.V) {
      set_status(p.status, TWELL_ERR_INDEX);
      id = -1;
    }
    if (v == -INFINITY) id = -1;
    te.id()[i] = id < 0 ? -1 : id;
    te.p[i] = v;
    te.z[i] = id >= 0 ? to_f(z[id]) : 0.f;
    any |= id >= 0;
  }
  for (int i = lane; i < DISTILL_MAX_K / 2; i += 32) te.seen4[i] = make_int4(-1, -1, -1, -1);
  __syncwarp();  // the list and the table before their readers (a vote orders no memory)
  return __any_sync(0xFFFFFFFFu, any);
}

// Its softmax, and for each id its first entry's sum, by the same warp.
__device__ __forceinline__ void list_softmax(Teacher &te, const DistillParams &p) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int i = lane; i < p.k; i += 32)
    if (te.id()[i] >= 0) m = fmaxf(m, te.p[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float sum = 0.f;
  for (int i = lane; i < p.k; i += 32)
    if (te.id()[i] >= 0) sum += ex2((te.p[i] - m) * p.c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  const float inv = 1.f / sum, ln = logf(sum);
  __syncwarp();
  for (int i = lane; i < p.k; i += 32) {
    const bool on = te.id()[i] >= 0;
    const float d = te.p[i] - m;
    te.p[i] = on ? ex2(d * p.c) * inv : 0.f;
    te.logp[i] = on ? d * p.inv_tau - ln : 0.f;
  }
  __syncwarp();
  // repeated ids (rare) are found by hashing; the warp sums each one's entries
  // in order (loss and gradient, 64 rows of 131072, k 128, one in a few rows: 12
  // us; where a lane went through the list for each of its entries 41)
  uint32_t again = 0;  // this lane's entries, one bit each
  for (int i = lane; i < p.k; i += 32) {
    const int id = te.id()[i];
    te.sum[i] = te.p[i];
    if (id < 0) continue;
    int *seen = (int *)te.seen4;
    unsigned h = ((unsigned)id * 2654435761u) >> 23;
    static_assert(DISTILL_MAX_K * 2 == 1 << (32 - 23), "the hash fills the table");
    for (;;) {
      const int old = atomicCAS(&seen[h], -1, id);
      if (old == id) again |= 1u << (i >> 5);
      if (old == -1 || old == id) break;
      h = (h + 1) % (2 * DISTILL_MAX_K);
    }
  }
  if (!__any_sync(0xFFFFFFFFu, again != 0)) return;
  __syncwarp();  // the lanes' sums before the other lanes read and change them
  for (int i0 = 0; i0 < p.k; i0 += 32) {
    uint32_t found = __ballot_sync(0xFFFFFFFFu, again >> (i0 >> 5) & 1);
    while (found) {
      const int i = i0 + __ffs(found) - 1, id = te.id()[i];
      found &= found - 1;
      if (te.sum[i] == -1.f) continue;  // (summed with another of its entries)
      __syncwarp();                     // (all have read it)
      float s = 0.f;
      int first = -1;
      for (int o = lane; o - lane < p.k; o += 32) {
        const bool same = o < p.k && te.id()[o] == id;
        uint32_t m = __ballot_sync(0xFFFFFFFFu, same);
        if (first < 0 && m) first = o - lane + __ffs(m) - 1;
        for (; m; m &= m - 1) s += te.p[o - lane + __ffs(m) - 1];
        if (same) te.sum[o] = -1.f;
      }
      __syncwarp();
      if (lane == 0) te.sum[first] = s;
      __syncwarp();
    }
  }
}

// The row's loss and statistics, by the same warp: m, l the maximum and the
// sum of exponentials, w the row's weight.
__device__ __forceinline__ void store_loss(Teacher &te, const DistillParams &p, size_t t, bool any,
                                           float w, float m, float l) {
  const int lane = threadIdx.x & 31;
  const Ref ref(m, p.c);
  const float log2l = log2f(l);
  float sum = 0.f;
  if (any)
    for (int i = lane; i < p.k; i += 32)
      if (te.id()[i] >= 0 && te.p[i] != 0.f)
        sum += te.p[i] * (te.logp[i] - (ref(te.z[i], p.c) - log2l) * LN2);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane != 0) return;
  p.loss[t] = any ? w * p.tau * p.tau * sum : 0.f;
  p.stats[t] = make_float2(m, logf(l) - (ref.wide ? 0.f : LN2 * fmaf(m, p.c, -ref.mc)));
}

// Gradient at the list's entries that the CTA owns, by the same warp after
// everything else there is written; gl = g / (sum of the exponentials).
template <typename E>
__device__ __forceinline__ void patch_entries(Teacher &te, const DistillParams &p,
                                              const Row<E> &row, E *out, int ja, int jb, bool first,
                                              const Ref &ref, float gl, float g) {
  for (int i = threadIdx.x & 31; i < p.k; i += 32) {
    const int id = te.id()[i];
    if (id >= 0 && row.owns(id, ja, jb, first) && !(te.sum[i] == -1.f))
      out[id] = from_f<E>(gl * ex2(ref(te.z[i], p.c)) - g * te.sum[i]);
  }
}

// Few rows: one cluster a row, each CTA a slice of `per` of its whole vectors
// (the first one the row's ends too).  The last warp keeps the teacher's list, the others
// stream.  GRAD: the first `cap` vectors of a slice stay in shared memory (all
// of them unless the row is longer than the cluster's shared memory; the rest
// is read again).
template <typename E, bool GRAD>
__global__ void __launch_bounds__(32 * (MAX_WARPS + 1), 3)
distill_forward_kernel(const E *z, E *dz, DistillParams p, int cap) {
  pdl_begin();
  constexpr int U = 4;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const size_t t = blockIdx.x / C;
  const E *zr = z + t * p.ldz;
  const Row<E> row(zr, p.V);
  E *out = GRAD ? dz + t * p.ldz : nullptr;
  const int per = (row.w1 - row.w0 + C - 1) / C;
  const int ja = min(row.w1, row.w0 + rank * per), jb = min(row.w1, ja + per);
  const bool first = rank == 0;
  // a masked row (uniform for the cluster) is not read: the weight is looked at
  // before the copies are issued, which costs the other rows nothing that shows
  // (us, with it first | behind the copies: 148 x 131072 bf16 25.1 | 24.5, 64 x
  // 131072 11.7 | 12.0; half the rows masked 17.0 | 19.3, 11.2 | 11.8)
  const float w = p.w ? p.w[t] : 1.f;
  if (w == 0.f) {
    if (GRAD) store_zeros(row, out, ja, jb, first, blockDim.x);
    if (first && threadIdx.x == 0) {
      p.loss[t] = 0.f;
      p.stats[t] = make_float2(0.f, 0.f);
    }
    return;
  }
  // [ja, js) go to shared memory, asynchronously and in two parts, before
  // anything is waited for (js: where it ends; jh: a multiple of the streaming
  // threads from ja on)
  extern __shared__ uint4 slice[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int SW = (int)blockDim.x / 32 - 1, ST = SW * 32;  // streaming warps, threads
  const int js = GRAD ? min(jb, ja + cap) : ja;
  const int jh = min(js, ja + ((js - ja) / 2 + ST - 1) / ST * ST);
  const uint64_t once = gather_policy<L2_FIRST>();
  if (GRAD && warp < SW) {
    for (int j = ja + (int)threadIdx.x; j < jh; j += ST) copy16_async(slice + (j - ja), row.base + j, once);
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (int j = jh + (int)threadIdx.x; j < js; j += ST) copy16_async(slice + (j - ja), row.base + j, once);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // (this CTA runs: its shared memory may be written by the others)
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  __shared__ Teacher te;
  __shared__ float2 s_part[MAX_CLUSTER * MAX_WARPS];  // (m, l) of the cluster's streaming warps
  __shared__ int s_any;
  const int e = first && warp < SW ? row.end(threadIdx.x) : -1;
  float ze = 0.f;  // this thread's end element

  float m = -INFINITY, l = 0.f;
  if (warp == SW) {
    const bool any = load_list(te, p, zr, t);
    if (lane == 0) s_any = any;
  } else {
    Running<E> sum(p.c);
    if (e >= 0) ze = to_f(zr[e]);
    if (!GRAD) {
      sum_vectors(sum, row, ja, jb, slice, ST, once);
    } else {  // what shared memory does not hold
      for (int j = js + (int)threadIdx.x; j < jb; j += U * ST) {
        uint4 r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j + u * ST < jb) r[u] = ld_once(row.base + j + u * ST);
        sum.add(r, jb - j, ST);
      }
    }
    if (GRAD) {  // (each thread reads back only what it copied)
      auto held = [&](int from, int to) {
        for (int j = from + (int)threadIdx.x; j < to; j += U * ST) {
          uint4 r[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (j + u * ST < to) r[u] = slice[j + u * ST - ja];
          sum.add(r, to - j, ST);
        }
      };
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      held(ja, jh);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      held(jh, js);
    }
    if (e >= 0) sum.add(ze);
    m = sum.m;
    l = sum.l;
    merge_warp(m, l, p.c);
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (warp < SW && lane < C)
    *cluster.map_shared_rank(&s_part[rank * SW + warp], lane) = make_float2(m, l);
  // (the last time that a CTA reaches into another, and, with a gradient in
  // place, that the row's logits are read by any but their owner)
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  if (warp == SW) list_softmax(te, p);
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  m = -INFINITY;
  l = 0.f;
  for (int i = lane; i < C * SW; i += 32) merge(m, l, s_part[i].x, s_part[i].y, p.c);
  merge_warp(m, l, p.c);
  const Ref ref(m, p.c);
  const bool any = s_any != 0;
  const float g = w * p.tau, gl = g / l;
  if (warp == SW) {
    if (first) store_loss(te, p, t, any, w, m, l);
  } else if (GRAD) {
    if (any) {
      uint4 *dst = (uint4 *)(out - row.lead);
      for (int j = ja + (int)threadIdx.x; j < jb; j += ST) {
        float f[VEC16<E>];
        grad_vec<E>(j < js ? slice[j - ja] : ld_once(row.base + j), ref, p.c, gl, f);
        stg_stream(dst + j, pack16(f, (E *)nullptr));
      }
      if (e >= 0) out[e] = from_f<E>(gl * ex2(ref(ze, p.c)));
    } else {
      store_zeros(row, out, ja, jb, first, ST);
    }
  }
  if (GRAD && any) {
    __syncthreads();  // all is written before the list's entries
    if (warp == SW) patch_entries(te, p, row, out, ja, jb, first, ref, gl, g);
  }
}

// Many rows: a CTA each, and with the gradient two streamed passes, the second
// one's reads from L2: at most 1024 streaming threads an SM keep 304 of the
// longest rows in flight (80 MB at 131072 bf16 logits; L2 has 126), and the
// first pass asks L2 to keep what it reads until the second has read it (206.5
// against 208 us at 2048 x 131072).  8192 x 131072, k 128: 0.75 ms, 5.7 TB/s, where
// the cluster kernel takes 1.04 ms: its CTAs stand still between reading and
// writing, and three of them an SM do not cover that.
template <typename E, int ROW_WARPS, bool GRAD>
__global__ void __launch_bounds__(32 * ROW_WARPS + 32, 1024 / (32 * ROW_WARPS))
distill_row_kernel(const E *z, E *dz, DistillParams p) {
  pdl_begin();
  constexpr int ROW_THREADS = 32 * ROW_WARPS;
  extern __shared__ uint4 slice[];  // the streaming threads' rings
  __shared__ Teacher te;
  __shared__ float2 s_part[ROW_WARPS];
  __shared__ int s_any;
  const size_t t = blockIdx.x;
  const E *zr = z + t * p.ldz;
  E *out = GRAD ? dz + t * p.ldz : nullptr;
  const Row<E> row(zr, p.V);
  const float w = p.w ? p.w[t] : 1.f;
  if (w == 0.f) {  // a masked row: nothing is read
    if (GRAD) store_zeros(row, out, row.w0, row.w1, true, blockDim.x);
    if (threadIdx.x == 0) {
      p.loss[t] = 0.f;
      p.stats[t] = make_float2(0.f, 0.f);
    }
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool lists = warp == ROW_WARPS;
  const int e = lists ? -1 : row.end(threadIdx.x);
  float ze = 0.f;
  if (lists) {
    const bool any = load_list(te, p, zr, t);
    if (lane == 0) s_any = any;
  } else {
    Running<E> sum(p.c);
    if (e >= 0) {
      ze = to_f(zr[e]);
      sum.add(ze);
    }
    sum_vectors(sum, row, row.w0, row.w1, slice, ROW_THREADS,
                GRAD ? keep_policy() : gather_policy<L2_FIRST>());
    merge_warp(sum.m, sum.l, p.c);
    if (lane == 0) s_part[warp] = make_float2(sum.m, sum.l);
  }
  __syncthreads();
  float m = lane < ROW_WARPS ? s_part[lane].x : -INFINITY;
  float l = lane < ROW_WARPS ? s_part[lane].y : 0.f;
  merge_warp(m, l, p.c);
  const Ref ref(m, p.c);
  const bool any = s_any != 0;
  const float g = w * p.tau, gl = g / l;
  if (lists) {
    if (any) list_softmax(te, p);
    store_loss(te, p, t, any, w, m, l);
  } else if (GRAD && any) {
    grad_vectors(row, out, row.w0, row.w1, slice, ROW_THREADS, ref, p.c, gl);
    if (e >= 0) out[e] = from_f<E>(gl * ex2(ref(ze, p.c)));
  } else if (GRAD) {
    store_zeros(row, out, row.w0, row.w1, true, ROW_THREADS);
  }
  if (!GRAD || !any) return;
  __syncthreads();  // all is written before the list's entries
  if (lists) patch_entries(te, p, row, out, row.w0, row.w1, true, ref, gl, g);
}

// The gradient from the forward's statistics: a row's slab of `slab_vecs`
// vectors a CTA, eight warps that stream and one for the list.
constexpr int BWD_THREADS = 256;

template <typename E>
__global__ void __launch_bounds__(BWD_THREADS + 32)
distill_backward_kernel(const E *z, E *dz, DistillParams p, int slabs, int slab_vecs) {
  pdl_begin();
  const size_t t = blockIdx.x / slabs;
  const E *zr = z + t * p.ldz;
  const Row<E> row(zr, p.V);
  E *out = dz + t * p.ldz;
  const int slab = (int)(blockIdx.x % slabs);
  const int ja = min(row.w1, row.w0 + slab * slab_vecs);
  const int jb = min(row.w1, ja + slab_vecs);
  const bool first = slab == 0;
  const float w = p.w[t];
  if (w == 0.f) {
    store_zeros(row, out, ja, jb, first, blockDim.x);
    return;
  }
  __shared__ Teacher te;
  __shared__ uint4 ring[RING * BWD_THREADS];
  const bool lists = threadIdx.x >= BWD_THREADS;
  // the row's list may be empty, so every warp looks at it
  bool used = false;
  for (int i = threadIdx.x & 31; i < p.k; i += 32) {
    const int id = p.ids[t * p.k + i];
    used |= id >= 0 && id < p.V && p.teacher[t * p.k + i] != -INFINITY;
  }
  const bool any = __any_sync(0xFFFFFFFFu, used);
  const float2 st = p.stats[t];
  const Ref ref(st.x, p.c);
  const float g = w * p.tau;
  const float gl = g * ex2(-st.y * LOG2E - (ref.wide ? 0.f : fmaf(st.x, p.c, -ref.mc)));
  if (lists) {
    // (with a gradient in place, the list's logits are read before the
    // barrier and overwritten after it; other CTAs write elsewhere, but may
    // be done with an entry's element already: only what this CTA owns is used)
    load_list(te, p, zr, t);
    __syncthreads();
    list_softmax(te, p);
  } else {
    __syncthreads();
    if (any) {
      grad_vectors(row, out, ja, jb, ring, BWD_THREADS, ref, p.c, gl);
      const int e = row.end(threadIdx.x);
      if (first && e >= 0) out[e] = from_f<E>(gl * ex2(ref(to_f(zr[e]), p.c)));
    } else {
      store_zeros(row, out, ja, jb, first, BWD_THREADS);
    }
  }
  __syncthreads();
  if (lists && any) patch_entries(te, p, row, out, ja, jb, first, ref, gl, g);
}

// Short rows: a warp each, which does it all; the second pass reads the row
// again from L1.
enum Pass { LOSS = 0, LOSS_GRAD = 1, GRAD_ONLY = 2 };
constexpr int SHORT_VECS = 256, SHORT_WARPS = 4;

template <typename E, int PASS>
__global__ void __launch_bounds__(SHORT_WARPS * 32)
distill_short_kernel(const E *z, E *dz, DistillParams p, int T) {
  pdl_begin();
  constexpr int N = VEC16<E>, U = 4;
  __shared__ Teacher lists[SHORT_WARPS];
  Teacher &te = lists[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const size_t t = (size_t)blockIdx.x * SHORT_WARPS + (threadIdx.x >> 5);
  if (t >= (size_t)T) return;
  const E *zr = z + t * p.ldz;
  const Row<E> row(zr, p.V);
  E *out = PASS == LOSS ? nullptr : dz + t * p.ldz;
  uint4 *dst = PASS == LOSS ? nullptr : (uint4 *)(out - row.lead);
  const int e = row.end(lane);
  const float w = p.w ? p.w[t] : 1.f;
  const bool any = w != 0.f && load_list(te, p, zr, t);
  if (w == 0.f && PASS != GRAD_ONLY && lane == 0) {
    p.loss[t] = 0.f;
    p.stats[t] = make_float2(0.f, 0.f);
  }
  const float ze = w != 0.f && e >= 0 ? to_f(zr[e]) : 0.f;
  float m = -INFINITY, l = 0.f, gl = 0.f;
  const float g = w * p.tau;
  if (w != 0.f && PASS != GRAD_ONLY) {
    Running<E> sum(p.c);
    for (int j = row.w0 + lane; j < row.w1; j += U * 32) {
      uint4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j + u * 32 < row.w1) r[u] = row.base[j + u * 32];
      sum.add(r, row.w1 - j, 32);
    }
    if (e >= 0) sum.add(ze);
    m = sum.m;
    l = sum.l;
    merge_warp(m, l, p.c);
    gl = g / l;
  }
  if (any) list_softmax(te, p);
  if (w != 0.f && PASS != GRAD_ONLY) store_loss(te, p, t, any, w, m, l);
  if (PASS == LOSS) return;
  if (!any) {  // masked, or a list of nothing
    for (int j = row.w0 + lane; j < row.w1; j += 32) dst[j] = make_uint4(0, 0, 0, 0);
    if (e >= 0) out[e] = from_f<E>(0.f);
    return;
  }
  if (PASS == GRAD_ONLY) {
    const float2 st = p.stats[t];
    const Ref ref(st.x, p.c);
    m = st.x;
    gl = g * ex2(-st.y * LOG2E - (ref.wide ? 0.f : fmaf(st.x, p.c, -ref.mc)));
  }
  const Ref ref(m, p.c);
  for (int j = row.w0 + lane; j < row.w1; j += 32) {
    float f[N];
    grad_vec<E>(row.base[j], ref, p.c, gl, f);
    dst[j] = pack16(f, (E *)nullptr);
  }
  if (e >= 0) out[e] = from_f<E>(gl * ex2(ref(ze, p.c)));
  __syncwarp();
  patch_entries(te, p, row, out, row.w0, row.w1, true, ref, gl, g);
}

DistillParams params_of(const DistillArgs &a) {
  DistillParams p;
  p.ids = a.ids; p.teacher = a.teacher; p.w = a.row_weight; p.ldz = a.ldz; p.V = a.V; p.k = a.k;
  p.tau = a.tau; p.c = LOG2E / a.tau; p.inv_tau = 1.f / a.tau;
  p.loss = a.loss; p.stats = (float2 *)a.stats; p.status = a.status;
  return p;
}

// Slices of at most 108 KB let two CTAs share an SM, so that one loads while
// the other writes (290 rows of 131072 | 200000 bf16 logits, us: 54 KB 45.1 | 68.5,
// 108 KB 43.4 | 67.2, 200 KB 59 | 82).
constexpr int SLICE_VECS = 108 * 1024 / 16, SLICE_MAX = 200 * 1024 / 16;

template <typename E, int PASS>
cudaError_t short_t(const DistillArgs &a, cudaStream_t s) {
  return launch_k(distill_short_kernel<E, PASS>,
                  dim3((unsigned)(((long long)a.T + SHORT_WARPS - 1) / SHORT_WARPS)),
                  dim3(SHORT_WARPS * 32), 0, s, (const E *)a.z, (E *)a.dz, params_of(a), a.T);
}

template <typename E, int ROW_WARPS, bool GRAD>
cudaError_t row_t(const DistillArgs &a, cudaStream_t s) {
  auto kern = distill_row_kernel<E, ROW_WARPS, GRAD>;
  constexpr int RING_BYTES = RING * 32 * ROW_WARPS * 16;
  static const cudaError_t attr =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BYTES);
  if (attr != cudaSuccess) return attr;
  return launch_k(kern, dim3((unsigned)a.T), dim3(32 * ROW_WARPS + 32), RING_BYTES, s,
                  (const E *)a.z, (E *)a.dz, params_of(a));
}

template <typename E, bool GRAD>
cudaError_t forward_t(const DistillArgs &a, cudaStream_t s) {
  if (a.V / VEC16<E> <= SHORT_VECS) return short_t<E, GRAD ? LOSS_GRAD : LOSS>(a, s);
  const int nvec = (int)((size_t)a.V / VEC16<E>);  // at most so many whole vectors
  // Streaming warps of a CTA, with the gradient, us at 8192 rows of 5001 | 12000 |
  // 32000 | 50001 | 80000 | 131072 bf16 logits, k 64: 4 warps 58 | 96 | 210 | 346 | 653
  // | 1072; 8 warps 88 | 118 | 206 | 280 | 536 | 1034; 16 warps 159 | 181 | 259 | 339 |
  // 472 | 743 (cluster kernel 102 | 139 | 263 | 413 | 706 | 1041).  The loss alone: 4
  // warps 39 | 52 | 87 | 123 | 203 | 327; 8 warps 56 | 67 | 99 | 133 | 205 | 325; 16 warps
  // 124 | 132 | 167 | 204 | 246 | 326 (cluster kernel 81 | 94 | 119 | 146 | 214 | 330): it
  // takes the same widths, which are not its best from 16384 to about 100000.
  // By rows, us at 5001 | 32000 | 131072 logits, cluster kernel and this rule's width:
  // 76 rows 6.9 | 7.5 | 15 and 6.0 | 8.2 | 17; 152 rows 6.7 | 8.2 | 26 and 6.5 | 8.4 | 17.5;
  // 256 rows 7.0 | 11.7 | 37 and 6.7 | 11.7 | 34; 304 rows 7.2 | 12.1 | 45 and 6.7 | 11.7 |
  // 37; 608 rows 8.8 | 22 | 84 and 7.4 | 18 | 73.
  if (a.T >= 2 * num_sms())
    return nvec <= 2048   ? row_t<E, 4, GRAD>(a, s)
           : nvec <= 7680 ? row_t<E, 8, GRAD>(a, s)
                          : row_t<E, 16, GRAD>(a, s);
  int C = 1;
  if (GRAD)
    while (C < MAX_CLUSTER && (nvec + C - 1) / C > SLICE_VECS) C *= 2;
  // few rows: split them until every SM has two CTAs or a slice is 16 KB (64 rows
  // of 50001, us: slices of 4 to 16 KB 8.8, 32 KB 7.4, 64 KB 7.8; one CTA an SM 7.3, four
  // 8.7; 64 and 148 rows of 131072 are the same within 2% throughout)
  while (C < MAX_CLUSTER && (long long)a.T * C < 2 * num_sms() && nvec / C >= 1024) C *= 2;
  const int per = (nvec + C - 1) / C;
  // (without a gradient: the ring of each streaming thread)
  const int cap = !GRAD ? RING * 32 * MAX_WARPS : per < SLICE_MAX ? per : SLICE_MAX;
  auto kern = distill_forward_kernel<E, GRAD>;
  static const cudaError_t attr =
      GRAD ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  SLICE_MAX * 16)
           : cudaSuccess;
  if (attr != cudaSuccess) return attr;
  if ((long long)a.T * C > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return launch_clusters(kern, dim3((unsigned)(a.T * C)), dim3(32 * (MAX_WARPS + 1)),
                         (size_t)cap * 16, C, s, (const E *)a.z, (E *)a.dz, params_of(a), cap);
}

template <typename E>
cudaError_t backward_t(const DistillArgs &a, cudaStream_t s) {
  if (a.V / VEC16<E> <= SHORT_VECS) return short_t<E, GRAD_ONLY>(a, s);
  const int nvec = a.V / VEC16<E>;
  // whole rows (the list is worked through once), in slabs of at least 1024
  // vectors while there are not four CTAs an SM (us, two | four | eight: 8 x 131072
  // 4.5 | 4.5 | 4.6, 64 x 131072 7.8 | 10.5 | 10.2, 300 x 50001 11.1 | 13.5 | 13.5, 600 x
  // 131072 53.8 | 52.3 | 52.0, 2048 x 50001 70 | 70 | 70; slabs of at least 512 and 2048
  // vectors: 8 x 50001 4.3 and 5.2, here 4.5)
  int slabs = 1;
  while ((long long)a.T * slabs < 4 * num_sms() && nvec / (2 * slabs) >= 1024) slabs *= 2;
  const int slab_vecs = (nvec + slabs - 1) / slabs;
  if ((long long)a.T * slabs > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return launch_k(distill_backward_kernel<E>, dim3((unsigned)((long long)a.T * slabs)),
                  dim3(BWD_THREADS + 32), 0, s, (const E *)a.z, (E *)a.dz, params_of(a), slabs, slab_vecs);
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
