// policy.cu -- clipped policy loss with a KL term: loss, gradient, and the
// log-probabilities alone.
//
//   logp = z[token] / tau - log sum exp(z / tau),  r = exp(logp - old),  d = ref - logp
//   loss = w (-min(r A, clip(r) A) + beta (exp(d) - d - 1)),  slope = d loss / d logp
//   dz = slope / tau (onehot - softmax(z / tau))
//
// As in the distillation loss the logits are the whole cost, and HBM bounds it: a row
// belongs to a warp (up to 256 vectors of 16 bytes), to a CTA that streams it twice, the
// second time from L2 (many rows: 8192 x 131072 bf16 with the gradient 708 us, 6.1 TB/s; the
// log-probabilities of 8192 x 50001 123 us, 6.7 TB/s), or to a cluster of CTAs that keep
// it in shared memory (few long rows).  What the row's scalars give is computed by every
// thread: the row's slope is known before its gradient is written, so no pass depends
// on another launch.
#include <cooperative_groups.h>

#include "common.cuh"
#include "lm_kernels.h"
#include "softmax_rows.cuh"

namespace cg = cooperative_groups;

namespace twell {

namespace {

constexpr int MAX_WARPS = 8;     // of a CTA of a cluster
constexpr int MAX_CLUSTER = 8;

struct PolicyParams {
  const void *tokens;
  int token_bytes;
  const float *old_logp, *ref_logp, *advantage, *w;
  long long ldz;
  int V;
  float c, inv_tau;  // c = log2(e) / tau
  float low, high, beta;  // the clip's ends, 1 - clip_low and 1 + clip_high
  float *loss, *logp;
  float2 *stats;
  int32_t *status;
};

// What stands beside a row's logits.
struct Token {
  int id;   // -1: the row is not read
  float w;
  __device__ __forceinline__ Token(const PolicyParams &p, size_t t) {
    w = p.w ? p.w[t] : 1.f;
    const long long k = p.token_bytes == 8 ? ((const long long *)p.tokens)[t]
                                           : (long long)((const int *)p.tokens)[t];
    id = w == 0.f || k < 0 || k >= p.V ? -1 : (int)k;
    if (k >= p.V && w != 0.f) set_status(p.status, TWELL_ERR_INDEX);
  }
};

// log-probability of a logit from the row's maximum and its sum of exponentials.
__device__ __forceinline__ float log_prob(float z, float m, float l, float c) {
  return (Ref(m, c)(z, c) - log2f(l)) * LN2;
}

// A factor of the gradient, held where its products with exponentials up to 2^(1/2), over sums
// of them from 2^(-1/2) on, are finite: an infinite one would make NaN of the elements of
// probability 0.
__device__ __forceinline__ float held(float v) {
  return v == v ? fminf(fmaxf(v, -0x1p126f), 0x1p126f) : v;
}

// The row's loss over its weight, and its slope over its weight.  Where exp(d) leaves fp32's
// range, so does the KL term (d, which may be infinite too, is not taken from it then).
__device__ __forceinline__ void row_loss(const PolicyParams &p, size_t t, float logp, float *loss,
                                         float *slope) {
  const float A = p.advantage[t];
  float r = logp == logp ? 1.f : logp;
  if (p.old_logp) r = expf(logp - p.old_logp[t]);
  // (infinity times 0 is 0 here; a NaN stays)
  const float gain = A == 0.f && r == INFINITY ? 0.f : r * A;
  const float kept = fminf(fmaxf(r, p.low), p.high) * A;
  const bool clipped = kept < gain;
  float l = -(clipped ? kept : gain), s = clipped ? 0.f : -held(gain);
  if (p.ref_logp && p.beta != 0.f) {
    const float d = p.ref_logp[t] - logp, e = expm1f(d);
    l += p.beta * (e == INFINITY ? e : e - d);
    s -= held(p.beta * e);
  }
  *loss = l;
  *slope = s;
}

// The gradient's factor of (onehot - softmax).
__device__ __forceinline__ float coef_of(const PolicyParams &p, const Token &tk, float slope) {
  return held(tk.w * slope * p.inv_tau);
}

// The row's outputs, by one thread; m, l: maximum and sum of exponentials.
// Returns the gradient's factor of (onehot - softmax).
__device__ __forceinline__ float finish_row(const PolicyParams &p, size_t t, const Token &tk,
                                            float zt, float m, float l, float *logp, bool store) {
  *logp = log_prob(zt, m, l, p.c);
  float loss = 0.f, slope = 0.f;
  if (p.advantage) row_loss(p, t, *logp, &loss, &slope);
  if (store) {
    const Ref ref(m, p.c);
    if (p.loss) p.loss[t] = tk.w * loss;
    p.logp[t] = *logp;
    p.stats[t] = make_float2(m, logf(l) - (ref.wide ? 0.f : LN2 * fmaf(m, p.c, -ref.mc)));
  }
  return coef_of(p, tk, slope);
}

__device__ __forceinline__ void store_nothing(const PolicyParams &p, size_t t) {
  if (p.loss) p.loss[t] = 0.f;
  p.logp[t] = 0.f;
  p.stats[t] = make_float2(0.f, 0.f);
}

// Gradient at the token (1 - q without cancellation).
template <typename E>
__device__ __forceinline__ void store_token(E *out, int id, float coef, float logp) {
  out[id] = from_f<E>(coef * -expm1f(logp));
}

// Few rows: one cluster a row, each CTA a slice of `per` of its whole vectors (the
// first one the row's ends too), of which with the gradient the first `cap` stay in
// shared memory.
template <typename E, bool GRAD>
__global__ void __launch_bounds__(32 * MAX_WARPS, 3)
policy_cluster_kernel(const E *z, E *dz, PolicyParams p, int cap) {
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
  const Token tk(p, t);
  if (tk.id < 0) {  // (the same for the whole cluster)
    if (GRAD) store_zeros(row, out, ja, jb, first, blockDim.x);
    if (first && threadIdx.x == 0) store_nothing(p, t);
    return;
  }
  extern __shared__ uint4 slice[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = (int)blockDim.x / 32, NT = W * 32;
  const int js = GRAD ? min(jb, ja + cap) : ja;
  const int jh = min(js, ja + ((js - ja) / 2 + NT - 1) / NT * NT);
  const uint64_t once = gather_policy<L2_FIRST>();
  if (GRAD) {
    for (int j = ja + (int)threadIdx.x; j < jh; j += NT) copy16_async(slice + (j - ja), row.base + j, once);
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (int j = jh + (int)threadIdx.x; j < js; j += NT) copy16_async(slice + (j - ja), row.base + j, once);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // (this CTA runs: its shared memory may be written by the others)
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  __shared__ float2 s_part[MAX_CLUSTER * MAX_WARPS];  // (m, l) of the cluster's warps
  const float zt = to_f(zr[tk.id]);
  const int e = first ? row.end(threadIdx.x) : -1;
  float ze = 0.f;  // this thread's end element
  Running<E> sum(p.c);
  if (e >= 0) ze = to_f(zr[e]);
  if (!GRAD) {
    sum_vectors(sum, row, ja, jb, slice, NT, once);
  } else {
    for (int j = js + (int)threadIdx.x; j < jb; j += U * NT) {  // what shared memory does not hold
      uint4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j + u * NT < jb) r[u] = ld_once(row.base + j + u * NT);
      sum.add(r, jb - j, NT);
    }
    auto held = [&](int from, int to) {  // (each thread reads back only what it copied)
      for (int j = from + (int)threadIdx.x; j < to; j += U * NT) {
        uint4 r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j + u * NT < to) r[u] = slice[j + u * NT - ja];
        sum.add(r, to - j, NT);
      }
    };
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    held(ja, jh);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    held(jh, js);
  }
  if (e >= 0) sum.add(ze);
  merge_warp(sum.m, sum.l, p.c);
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (lane < C)
    *cluster.map_shared_rank(&s_part[rank * W + warp], lane) = make_float2(sum.m, sum.l);
  // (the last time that a CTA reaches into another, and, with a gradient in
  // place, that the row's logits are read by any but their owner)
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  float m = -INFINITY, l = 0.f;
  for (int i = lane; i < C * W; i += 32) merge(m, l, s_part[i].x, s_part[i].y, p.c);
  merge_warp(m, l, p.c);
  float logp;
  const float coef = finish_row(p, t, tk, zt, m, l, &logp, first && threadIdx.x == 0);
  if (!GRAD) return;
  const Ref ref(m, p.c);
  const float gl = -coef / l;
  uint4 *dst = (uint4 *)(out - row.lead);
  for (int j = ja + (int)threadIdx.x; j < jb; j += NT) {
    float f[VEC16<E>];
    grad_vec<E>(j < js ? slice[j - ja] : ld_once(row.base + j), ref, p.c, gl, f);
    stg_stream(dst + j, pack16(f, (E *)nullptr));
  }
  if (e >= 0) out[e] = from_f<E>(gl * ex2(ref(ze, p.c)));
  __syncthreads();  // all is written before the token's element
  if (threadIdx.x == 0 && row.owns(tk.id, ja, jb, first)) store_token(out, tk.id, coef, logp);
}

// Many rows: a CTA each, and with the gradient two streamed passes, the second
// one's reads from L2.
template <typename E, int ROW_WARPS, bool GRAD>
__global__ void __launch_bounds__(32 * ROW_WARPS, 1024 / (32 * ROW_WARPS))
policy_row_kernel(const E *z, E *dz, PolicyParams p) {
  pdl_begin();
  constexpr int NT = 32 * ROW_WARPS;
  extern __shared__ uint4 ring[];
  __shared__ float2 s_part[ROW_WARPS];
  const size_t t = blockIdx.x;
  const E *zr = z + t * p.ldz;
  E *out = GRAD ? dz + t * p.ldz : nullptr;
  const Row<E> row(zr, p.V);
  const Token tk(p, t);
  if (tk.id < 0) {
    if (GRAD) store_zeros(row, out, row.w0, row.w1, true, NT);
    if (threadIdx.x == 0) store_nothing(p, t);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = row.end(threadIdx.x);
  const float zt = to_f(zr[tk.id]);
  Running<E> sum(p.c);
  float ze = 0.f;
  if (e >= 0) {
    ze = to_f(zr[e]);
    sum.add(ze);
  }
  sum_vectors(sum, row, row.w0, row.w1, ring, NT, GRAD ? keep_policy() : gather_policy<L2_FIRST>());
  merge_warp(sum.m, sum.l, p.c);
  if (lane == 0) s_part[warp] = make_float2(sum.m, sum.l);
  __syncthreads();
  float m = lane < ROW_WARPS ? s_part[lane].x : -INFINITY;
  float l = lane < ROW_WARPS ? s_part[lane].y : 0.f;
  merge_warp(m, l, p.c);
  float logp;
  const float coef = finish_row(p, t, tk, zt, m, l, &logp, threadIdx.x == 0);
  if (!GRAD) return;
  const Ref ref(m, p.c);
  const float gl = -coef / l;
  grad_vectors(row, out, row.w0, row.w1, ring, NT, ref, p.c, gl);
  if (e >= 0) out[e] = from_f<E>(gl * ex2(ref(ze, p.c)));
  __syncthreads();  // all is written before the token's element
  if (threadIdx.x == 0) store_token(out, tk.id, coef, logp);
}

// The gradient from the forward's statistics: a row's slab of `slab_vecs` vectors
// a CTA.
constexpr int BWD_THREADS = 256;

// The same from the statistics, and that of the exponentials.
__device__ __forceinline__ float coef_of(const PolicyParams &p, size_t t, const Token &tk,
                                         float logp) {
  float loss, slope;
  row_loss(p, t, logp, &loss, &slope);
  return coef_of(p, tk, slope);
}
__device__ __forceinline__ float gl_of(float coef, const float2 &st, const Ref &ref, float c) {
  return -coef * ex2(-st.y * LOG2E - (ref.wide ? 0.f : fmaf(st.x, c, -ref.mc)));
}

template <typename E>
__global__ void __launch_bounds__(BWD_THREADS)
policy_backward_kernel(const E *z, E *dz, PolicyParams p, int slabs, int slab_vecs) {
  pdl_begin();
  __shared__ uint4 ring[RING * BWD_THREADS];
  const size_t t = blockIdx.x / slabs;
  const E *zr = z + t * p.ldz;
  const Row<E> row(zr, p.V);
  E *out = dz + t * p.ldz;
  const int slab = (int)(blockIdx.x % slabs);
  const int ja = min(row.w1, row.w0 + slab * slab_vecs);
  const int jb = min(row.w1, ja + slab_vecs);
  const bool first = slab == 0;
  const Token tk(p, t);
  if (tk.id < 0) {
    store_zeros(row, out, ja, jb, first, BWD_THREADS);
    return;
  }
  const float2 st = p.stats[t];
  const float logp = p.logp[t], coef = coef_of(p, t, tk, logp);
  const Ref ref(st.x, p.c);
  const float gl = gl_of(coef, st, ref, p.c);
  grad_vectors(row, out, ja, jb, ring, BWD_THREADS, ref, p.c, gl);
  const int e = row.end(threadIdx.x);
  if (first && e >= 0) out[e] = from_f<E>(gl * ex2(ref(to_f(zr[e]), p.c)));
  __syncthreads();
  if (threadIdx.x == 0 && row.owns(tk.id, ja, jb, first)) store_token(out, tk.id, coef, logp);
}

// Short rows: a warp each; the second pass reads the row again from L1.
enum Pass { LOSS = 0, LOSS_GRAD = 1, GRAD_ONLY = 2 };
constexpr int SHORT_VECS = 256, SHORT_WARPS = 4;

template <typename E, int PASS>
__global__ void __launch_bounds__(SHORT_WARPS * 32)
policy_short_kernel(const E *z, E *dz, PolicyParams p, int T) {
  pdl_begin();
  constexpr int N = VEC16<E>, U = 4;
  const int lane = threadIdx.x & 31;
  const size_t t = (size_t)blockIdx.x * SHORT_WARPS + (threadIdx.x >> 5);
  if (t >= (size_t)T) return;
  const E *zr = z + t * p.ldz;
  const Row<E> row(zr, p.V);
  E *out = PASS == LOSS ? nullptr : dz + t * p.ldz;
  uint4 *dst = PASS == LOSS ? nullptr : (uint4 *)(out - row.lead);
  const int e = row.end(lane);
  const Token tk(p, t);
  if (tk.id < 0) {
    if (PASS != GRAD_ONLY && lane == 0) store_nothing(p, t);
    if (PASS == LOSS) return;
    for (int j = row.w0 + lane; j < row.w1; j += 32) dst[j] = make_uint4(0, 0, 0, 0);
    if (e >= 0) out[e] = from_f<E>(0.f);
    return;
  }
  const float ze = e >= 0 ? to_f(zr[e]) : 0.f;
  float m, l = 1.f, logp, coef, gl = 0.f;
  if (PASS != GRAD_ONLY) {
    const float zt = to_f(zr[tk.id]);
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
    coef = finish_row(p, t, tk, zt, m, l, &logp, lane == 0);
    gl = -coef / l;
  } else {
    const float2 st = p.stats[t];
    m = st.x;
    logp = p.logp[t];
    coef = coef_of(p, t, tk, logp);
    gl = gl_of(coef, st, Ref(m, p.c), p.c);
  }
  if (PASS == LOSS) return;
  const Ref ref(m, p.c);
  __syncwarp();  // (in place: the token's logit is read by all lanes before it is overwritten)
  for (int j = row.w0 + lane; j < row.w1; j += 32) {
    float f[N];
    grad_vec<E>(row.base[j], ref, p.c, gl, f);
    dst[j] = pack16(f, (E *)nullptr);
  }
  if (e >= 0) out[e] = from_f<E>(gl * ex2(ref(ze, p.c)));
  __syncwarp();
  if (lane == 0) store_token(out, tk.id, coef, logp);
}

PolicyParams params_of(const PolicyArgs &a) {
  PolicyParams p;
  p.tokens = a.tokens; p.token_bytes = a.token_bytes; p.old_logp = a.old_logp;
  p.ref_logp = a.ref_logp; p.advantage = a.advantage; p.w = a.row_weight; p.ldz = a.ldz; p.V = a.V;
  p.c = LOG2E / a.tau; p.inv_tau = 1.f / a.tau;
  p.low = 1.f - a.clip_low; p.high = 1.f + a.clip_high; p.beta = a.beta;
  p.loss = a.loss; p.logp = a.logp; p.stats = (float2 *)a.stats; p.status = a.status;
  return p;
}

// Slices of at most 108 KB let two CTAs share an SM, so that one loads while the
// other writes.
constexpr int SLICE_VECS = 108 * 1024 / 16, SLICE_MAX = 200 * 1024 / 16;

template <typename E, int PASS>
cudaError_t short_t(const PolicyArgs &a, cudaStream_t s) {
  return launch_k(policy_short_kernel<E, PASS>,
                  dim3((unsigned)(((long long)a.T + SHORT_WARPS - 1) / SHORT_WARPS)),
                  dim3(SHORT_WARPS * 32), 0, s, (const E *)a.z, (E *)a.dz, params_of(a), a.T);
}

template <typename E, int ROW_WARPS, bool GRAD>
cudaError_t row_t(const PolicyArgs &a, cudaStream_t s) {
  auto kern = policy_row_kernel<E, ROW_WARPS, GRAD>;
  constexpr int RING_BYTES = RING * 32 * ROW_WARPS * 16;
  static const cudaError_t attr =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BYTES);
  if (attr != cudaSuccess) return attr;
  return launch_k(kern, dim3((unsigned)a.T), dim3(32 * ROW_WARPS), RING_BYTES, s, (const E *)a.z,
                  (E *)a.dz, params_of(a));
}

// Warps of a row's CTA, 0 for clusters.  us of the cluster kernel | 4 | 8 | 16 warps,
// with the gradient, at 12000, 50001 and 131072 bf16 logits:
//   8192 rows  105|71|93|151    387|351|274|336   834|930|894|709
//   2048        30|23|25|38     105|92|80|91      216|244|226|187
//   304        7.0|6.1|5.6|6.2   18|18|17|17       39|39|34|32
//   152        5.6|5.4|4.5|4.5   11|14|12|11       24|29|20|18
//   64         5.0|5.0|4.1|4.2  8.8|13|10|9.3      12|28|19|15
// and the log-probabilities alone:
//   8192        70|39|47|71     145|123|130|149   305|306|300|312
//   2048        20|13|14|20      41|40|37|41       84|92|82|84
//   304        4.6|4.0|3.6|4.1  9.6|9.7|8.6|9.2    17|19|15|16
//   152        3.9|3.4|2.9|2.9  7.2|8.5|6.5|6.1    11|17|12|9.7
//   64         3.6|3.3|2.8|2.8  5.6|8.1|6.0|5.4   8.4|16|11|8.6
// (With few rows, a row's latency counts; with many, that the rows in flight fit into L2
// and the warps into the SMs.)
// fp32 goes by the same vectors: with the gradient at 6000, 12000, 50001 and 131072 logits
//   8192 rows   91|67|84|137    137|129|134|171    614|748|678|551   1532|1851|1824|1770
//   304        6.7|5.3|5.0|5.4   10|9.4|8.6|8.4     31|32|30|29       66|79|72|70
//   64         4.7|4.4|3.7|3.8  5.2|6.2|4.9|4.5    9.9|20|16|14       22|41|29|22
// and alone
//   8192        60|30|36|60      76|57|56|72       229|234|230|223    570|587|579|566
//   304        4.5|3.6|3.3|3.5  6.3|5.3|5.0|5.0     14|14|13|13       26|29|24|25
//   64         3.4|2.9|2.5|2.5  3.6|4.1|3.1|2.8    6.6|12|7.7|6.2    9.5|26|15|10
// so the rule's choice is the best or within a tenth of it, but for many rows of 512 KB with
// the gradient, where clusters would read less from HBM twice.
int row_warps(long long rows, int nvec, bool grad) {
  const int sms = num_sms();
  const bool short_ = nvec <= 2048;  // 32 KB
  if (rows >= 2 * sms) {
    if (short_) return rows >= 4 * sms ? 4 : 8;
    if (grad) return nvec <= 7680 ? 8 : 16;
    return rows >= 48 * sms && nvec <= 10240 ? 4 : 8;
  }
  if (short_) return 8;
  if (rows >= sms) return 16;
  return !grad && rows >= sms / 4 && nvec <= 10240 ? 16 : 0;
}

template <typename E, bool GRAD>
cudaError_t forward_t(const PolicyArgs &a, cudaStream_t s) {
  if (a.V / VEC16<E> <= SHORT_VECS) return short_t<E, GRAD ? LOSS_GRAD : LOSS>(a, s);
  const int nvec = (int)((size_t)a.V / VEC16<E>);  // at most so many whole vectors
  switch (row_warps(a.T, nvec, GRAD)) {
    case 4: return row_t<E, 4, GRAD>(a, s);
    case 8: return row_t<E, 8, GRAD>(a, s);
    case 16: return row_t<E, 16, GRAD>(a, s);
  }
  int C = 1;
  if (GRAD)
    while (C < MAX_CLUSTER && (nvec + C - 1) / C > SLICE_VECS) C *= 2;
  // few rows: split them until every SM has two CTAs or a slice is 16 KB
  while (C < MAX_CLUSTER && (long long)a.T * C < 2 * num_sms() && nvec / C >= 1024) C *= 2;
  const int per = (nvec + C - 1) / C;
  // (without a gradient: the ring of each thread)
  const int cap = !GRAD ? RING * 32 * MAX_WARPS : per < SLICE_MAX ? per : SLICE_MAX;
  auto kern = policy_cluster_kernel<E, GRAD>;
  static const cudaError_t attr =
      GRAD ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  SLICE_MAX * 16)
           : cudaSuccess;
  if (attr != cudaSuccess) return attr;
  return launch_clusters(kern, dim3((unsigned)(a.T * C)), dim3(32 * MAX_WARPS), (size_t)cap * 16, C,
                         s, (const E *)a.z, (E *)a.dz, params_of(a), cap);
}

template <typename E>
cudaError_t backward_t(const PolicyArgs &a, cudaStream_t s) {
  if (a.V / VEC16<E> <= SHORT_VECS) return short_t<E, GRAD_ONLY>(a, s);
  const int nvec = a.V / VEC16<E>;
  // whole rows, in slabs of at least 1024 vectors while there are not four CTAs an SM (us,
  // two | four | eight: 64 x 131072 7.0 | 7.5 | 7.5, 152 x 131072 14.1 | 13.6 | 13.6, 304 x
  // 50001 11.7 | 11.5 | 11.6, 2048 rows and more the same)
  int slabs = 1;
  while ((long long)a.T * slabs < 4 * num_sms() && nvec / (2 * slabs) >= 1024) slabs *= 2;
  const int slab_vecs = (nvec + slabs - 1) / slabs;
  return launch_k(policy_backward_kernel<E>, dim3((unsigned)((long long)a.T * slabs)),
                  dim3(BWD_THREADS), 0, s, (const E *)a.z, (E *)a.dz, params_of(a), slabs,
                  slab_vecs);
}

}  // namespace

cudaError_t launch_policy_forward(const PolicyArgs &a, cudaStream_t s) {
  if (a.dtype == TWELL_BF16) return a.dz ? forward_t<bf16, true>(a, s) : forward_t<bf16, false>(a, s);
  return a.dz ? forward_t<float, true>(a, s) : forward_t<float, false>(a, s);
}

cudaError_t launch_policy_backward(const PolicyArgs &a, cudaStream_t s) {
  return a.dtype == TWELL_BF16 ? backward_t<bf16>(a, s) : backward_t<float>(a, s);
}

}  // namespace twell
