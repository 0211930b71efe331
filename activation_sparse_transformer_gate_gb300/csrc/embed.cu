// embed.cu -- token embedding with scaling, and its gradient by sorted tokens.
//
// forward   out[t] = scale E[tok_t]
// gradient  dE[v]  = scale sum_{t: tok_t = v} dy[t]
//
// Both move rows and add; HBM bounds them.  The gradient writes the whole
// [V][D] fp32 table once and reads dy once (V 131072, D 4096, 16384 tokens at
// random: 347 us, 6.6 TB/s).  A gather per row in a fixed
// order needs the positions grouped by token, so:
//   1. one launch sorts (token, position) -- a stable radix sort by one
//      thread-block cluster, or by one CTA -- while every other CTA writes the
//      zeros of the table;
//   2. the sorted list is cut into equal chunks, so that reading dy is spread
//      evenly whatever the tokens are: a run of equal tokens inside a chunk is
//      summed and stored, a run that crosses a chunk's end leaves its part in
//      the workspace;
//   3. the parts of each crossing run are added in order: one part a chunk, so
//      this grows with the longest run (D 2048, V 50001: 16384 tokens 94 us, half
//      of them one token 111; 131072 tokens 336 and 504).
// Up to 512 tokens one launch compares the positions instead.  No
// floating-point atomics: the grouping of every sum is fixed by T and the tokens
// alone.
#include <cooperative_groups.h>

#include "common.cuh"
#include "lm_kernels.h"
#include "vec16.cuh"

namespace cg = cooperative_groups;

namespace twell {

namespace {

constexpr int SORT_CTAS = 8;       // CTAs of the sorting cluster (the portable maximum)
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int DIGIT_MAX = 9;       // bits per pass: 2 passes sort any vocabulary below 2^18
constexpr int ZERO_VECS = 2048;    // 16-byte vectors that a CTA zeroes
constexpr int CHUNK = 16;          // sorted entries per chunk of step 2

// The token at position t as a sort key: the token, or V for positions
// without one (padding, or out of range: recorded).
template <typename I>
__device__ __forceinline__ uint32_t token_key(const I *tokens, int t, int V, long long pad_id,
                                              int32_t *status) {
  const long long v = (long long)tokens[t];
  if (v == pad_id) return (uint32_t)V;
  if (v < 0 || v >= V) {
    set_status(status, TWELL_ERR_INDEX);
    return (uint32_t)V;
  }
  return (uint32_t)v;
}

// One warp per 128 vectors (2 KB) of a row, four independent loads a lane.
template <typename E, typename I>
__global__ void __launch_bounds__(256)
embed_forward_kernel(const I *tokens, const E *table, int T, int V, int nv, float scale,
                     long long pad_id, E *out, int32_t *status) {
  pdl_begin();
  constexpr int N = VEC16<E>;
  const int parts = (nv + 127) / 128;
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long t = unit / parts;
  if (t >= T) return;
  const int v0 = (int)(unit - t * parts) * 128 + (threadIdx.x & 31);
  const uint32_t key = token_key(tokens, (int)t, V, pad_id, status);
  const bool live = key < (uint32_t)V;
  const uint4 *src = (const uint4 *)table + (size_t)(live ? key : 0) * nv;
  uint4 *dst = (uint4 *)out + (size_t)t * nv;
  uint4 r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = live && v0 + 32 * i < nv ? ldg_stream(src + v0 + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (v0 + 32 * i >= nv) break;
    float f[N];
    unpack(r[i], f, (E *)nullptr);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] *= scale;
    stg_stream(dst + v0 + 32 * i, live ? pack16(f, (E *)nullptr) : make_uint4(0, 0, 0, 0));
  }
}

// ---- step 1: sort and zero ---------------------------------------------------
// Cluster 0 sorts; each CTA of the other clusters zeroes one 32 KB piece (as
// few long-lived CTAs, of which not all fitted at once, the zeros took 492
// where they now take 275 us for 2.1 GB).  Least
// significant digit first; each CTA owns a contiguous eighth of the list and
// each warp a contiguous part of that, walked in order, so that (digit, CTA,
// warp, place in the warp's walk) is the stable order.  Per pass: counts per
// warp and digit in shared memory, the CTAs' totals exchanged through
// distributed shared memory, then every key is stored at its place.
__device__ __forceinline__ void zero_piece(uint4 *dtable, size_t table_vecs, int piece) {
  const size_t i0 = (size_t)piece * ZERO_VECS + threadIdx.x;
#pragma unroll
  for (int i = 0; i < ZERO_VECS; i += SORT_THREADS)
    if (i0 + i < table_vecs) dtable[i0 + i] = make_uint4(0, 0, 0, 0);
}

struct SortSmem {
  uint32_t hist[SORT_WARPS][1 << DIGIT_MAX];  // counts, then each warp's next place
  uint32_t total[1 << DIGIT_MAX];             // this CTA's count per digit
  uint32_t warp_sum[SORT_WARPS];
};

template <typename I>
__global__ void __launch_bounds__(SORT_THREADS, 2)
embed_sort_zero_kernel(const I *tokens, int T, int V, long long pad_id, uint32_t *key0,
                       int32_t *pos0, uint32_t *key1, int32_t *pos1, int passes, int bits,
                       uint4 *dtable, size_t table_vecs, int32_t *status) {
  pdl_begin();
  if (blockIdx.x >= SORT_CTAS) {
    zero_piece(dtable, table_vecs, (int)blockIdx.x - SORT_CTAS);
    return;
  }
  extern __shared__ uint8_t sort_smem_raw[];
  SortSmem &sm = *(SortSmem *)sort_smem_raw;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bins = 1 << bits;
  // this warp's part of the list, in groups of 32
  const long long groups = ((long long)T + 31) / 32;
  const long long warps = (long long)SORT_CTAS * SORT_WARPS;
  const long long w = (long long)rank * SORT_WARPS + warp;
  const long long g0 = groups * w / warps, g1 = groups * (w + 1) / warps;

  for (int pass = 0; pass < passes; ++pass) {
    // (the last pass ends in key0 / pos0 whatever their number)
    const bool to0 = ((passes - 1 - pass) & 1) == 0;
    const uint32_t *kin = to0 ? key1 : key0;
    const int32_t *pin = to0 ? pos1 : pos0;
    uint32_t *kout = to0 ? key0 : key1;
    int32_t *pout = to0 ? pos0 : pos1;
    const int shift = pass * bits;
    auto load = [&](long long i) -> uint32_t {
      if (i >= T) return 0xFFFFFFFFu;
      return pass == 0 ? token_key(tokens, (int)i, V, pad_id, status) : __ldcg(kin + i);
    };
    for (int b = lane; b < bins; b += 32) sm.hist[warp][b] = 0;
    __syncwarp();
    for (long long g = g0; g < g1; ++g) {
      const long long i = g * 32 + lane;
      const uint32_t k = load(i);
      const uint32_t d = i < T ? (k >> shift) & (bins - 1) : 0xFFFFFFFFu;
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, d);
      if (i < T && lane == __ffs(peers) - 1) sm.hist[warp][d] += __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    // each digit: the warps' counts become offsets within the CTA
    if (threadIdx.x < bins) {
      uint32_t run = 0;
      for (int i = 0; i < SORT_WARPS; ++i) {
        const uint32_t c = sm.hist[i][threadIdx.x];
        sm.hist[i][threadIdx.x] = run;
        run += c;
      }
      sm.total[threadIdx.x] = run;
    }
    cluster.sync();
    uint32_t before = 0, all = 0;
    if (threadIdx.x < bins)
      for (int c = 0; c < SORT_CTAS; ++c) {
        const uint32_t n = *cluster.map_shared_rank(&sm.total[threadIdx.x], c);
        if (c < rank) before += n;
        all += n;
      }
    // exclusive scan of the digits' totals
    uint32_t inc = all;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) sm.warp_sum[warp] = inc;
    __syncthreads();
    if (threadIdx.x < bins) {
      uint32_t base = inc - all + before;
      for (int i = 0; i < warp; ++i) base += sm.warp_sum[i];
      for (int i = 0; i < SORT_WARPS; ++i) sm.hist[i][threadIdx.x] += base;
    }
    __syncthreads();
    for (long long g = g0; g < g1; ++g) {
      const long long i = g * 32 + lane;
      const uint32_t k = load(i);
      const uint32_t d = i < T ? (k >> shift) & (bins - 1) : 0xFFFFFFFFu;
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, d);
      if (i < T) {
        const uint32_t to = sm.hist[warp][d] + __popc(peers & ((1u << lane) - 1));
        kout[to] = k;
        pout[to] = pass == 0 ? (int32_t)i : __ldcg(pin + i);
      }
      __syncwarp();
      if (i < T && lane == __ffs(peers) - 1) sm.hist[warp][d] += __popc(peers);
      __syncwarp();
    }
    // the pass's stores reach the other CTAs, and no CTA's totals are
    // overwritten (or its shared memory freed) while another reads them
    __threadfence();
    cluster.sync();
  }
}

// The same sort for up to ALONE tokens below 2^18 by CTA 0 alone, while the
// others zero: the keys stay in registers and, between the two passes, in shared
// memory, and a key's place in its warp's walk is kept from the counting.  The
// gradient's us, alone | by the cluster: 513 tokens, V 1000, D 256 9.9 | 13.3; 1000
// tokens 10.9 | 12.7; 2000 tokens, V 8192, D 512 15.1 | 15.9; with eight groups a
// warp 4096 tokens 20.4 | 17.6.
constexpr int ALONE_GROUPS = 4;  // of 32 tokens, a warp
constexpr int ALONE = SORT_WARPS * 32 * ALONE_GROUPS;
struct AloneSmem {
  SortSmem sort;
  uint32_t key[ALONE];
  uint16_t pos[ALONE];
};

template <typename I>
__global__ void __launch_bounds__(SORT_THREADS, 2)
embed_alone_zero_kernel(const I *tokens, int T, int V, long long pad_id, uint32_t *key,
                        int32_t *pos, int passes, int bits, uint4 *dtable, size_t table_vecs,
                        int32_t *status) {
  pdl_begin();
  if (blockIdx.x > 0) {
    zero_piece(dtable, table_vecs, (int)blockIdx.x - 1);
    return;
  }
  extern __shared__ uint8_t sort_smem_raw[];
  AloneSmem &am = *(AloneSmem *)sort_smem_raw;
  SortSmem &sm = am.sort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bins = 1 << bits;
  const int groups = (T + 31) / 32;
  const int g0 = groups * warp / SORT_WARPS, g1 = groups * (warp + 1) / SORT_WARPS;
  for (int pass = 0; pass < passes; ++pass) {
    const bool last = pass == passes - 1;
    const int shift = pass * bits;
    uint32_t k[ALONE_GROUPS], at[ALONE_GROUPS];
    int from[ALONE_GROUPS];
#pragma unroll
    for (int j = 0; j < ALONE_GROUPS; ++j) {
      const int i = (g0 + j) * 32 + lane;
      const bool live = g0 + j < g1 && i < T;
      k[j] = !live ? 0u : pass == 0 ? token_key(tokens, i, V, pad_id, status) : am.key[i];
      from[j] = !live ? -1 : pass == 0 ? i : am.pos[i];
    }
    for (int b = lane; b < bins; b += 32) sm.hist[warp][b] = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < ALONE_GROUPS; ++j) {
      if (g0 + j >= g1) break;
      const uint32_t d = from[j] >= 0 ? (k[j] >> shift) & (bins - 1) : 0xFFFFFFFFu;
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, d);
      const uint32_t before = from[j] >= 0 ? sm.hist[warp][d] : 0;
      at[j] = before + __popc(peers & ((1u << lane) - 1));
      __syncwarp();
      if (from[j] >= 0 && lane == __ffs(peers) - 1) sm.hist[warp][d] = before + __popc(peers);
      __syncwarp();
    }
    __syncthreads();  // (all have read their keys too)
    // each digit: the warps' counts become places
    uint32_t c[SORT_WARPS], all = 0;
    if (threadIdx.x < bins) {
#pragma unroll
      for (int i = 0; i < SORT_WARPS; ++i) c[i] = sm.hist[i][threadIdx.x];
#pragma unroll
      for (int i = 0; i < SORT_WARPS; ++i) all += c[i];
    }
    uint32_t inc = all;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) sm.warp_sum[warp] = inc;
    __syncthreads();
    if (threadIdx.x < bins) {
      uint32_t run = inc - all;
      for (int i = 0; i < warp; ++i) run += sm.warp_sum[i];
#pragma unroll
      for (int i = 0; i < SORT_WARPS; ++i) {
        sm.hist[i][threadIdx.x] = run;
        run += c[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ALONE_GROUPS; ++j) {
      if (from[j] < 0) continue;
      const uint32_t to = sm.hist[warp][(k[j] >> shift) & (bins - 1)] + at[j];
      if (last) {
        key[to] = k[j];
        pos[to] = from[j];
      } else {
        am.key[to] = k[j];
        am.pos[to] = (uint16_t)from[j];
      }
    }
    __syncthreads();
  }
}

// ---- step 2: runs of equal tokens --------------------------------------------
// A group of `tpr` threads (whole warps) takes one chunk and one slab of tpr
// 16-byte vectors.  Every warp holds the chunk's keys and positions a lane
// each; rows are loaded eight at a time ahead of their use.
template <typename E>
__global__ void __launch_bounds__(256)
embed_runs_kernel(const uint32_t *key, const int32_t *pos, const E *dy, int T, int V, int nv,
                  int tpr, int chunks, float scale, float *dtable, float *part) {
  pdl_begin();
  constexpr int N = VEC16<E>, U = 8;
  static_assert(CHUNK + 2 <= 32, "a warp holds a chunk and its neighbours");
  const int c = (int)blockIdx.x * (blockDim.x / tpr) + (int)threadIdx.x / tpr;
  const int v = (int)blockIdx.y * tpr + (int)threadIdx.x % tpr;
  if (c >= chunks) return;  // (uniform for the warp)
  const int lane = threadIdx.x & 31;
  const int i0 = c * CHUNK, n = min(T - i0, CHUNK);
  const int D = nv * N;
  // lane 0: the entry before the chunk; 1 .. n: the chunk; n + 1: the next
  const int at = i0 + lane - 1;
  const uint32_t NONE = 0xFFFFFFFFu;
  const uint32_t k_of = at >= 0 && at < T && lane <= n + 1 ? key[at] : NONE;
  const int p_of = lane >= 1 && lane <= n ? pos[at] : 0;
  // the chunk's first run began before it / its last run goes on after it
  bool left = __shfl_sync(NONE, k_of, 0) == __shfl_sync(NONE, k_of, 1);
  const bool open_right = __shfl_sync(NONE, k_of, n) == __shfl_sync(NONE, k_of, n + 1);
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.f;
  for (int i = 0; i < n; i += U) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t k = __shfl_sync(NONE, k_of, min(i + u, CHUNK) + 1);
      const int p = __shfl_sync(NONE, p_of, min(i + u, CHUNK) + 1);
      r[u] = i + u < n && k < (uint32_t)V && v < nv ? ldg_stream((const uint4 *)dy + (size_t)p * nv + v)
                                                    : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t k = __shfl_sync(NONE, k_of, min(i + u, CHUNK) + 1);
      const uint32_t next = __shfl_sync(NONE, k_of, min(i + u + 1, CHUNK) + 1);
      if (i + u >= n || k >= (uint32_t)V) continue;  // no token here, nor further on
      float f[N];
      unpack(r[u], f, (E *)nullptr);
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] += f[j];
      if (i + u + 1 < n && next == k) continue;
      // the run ends with this entry (or the chunk does)
      const bool right = open_right && i + u == n - 1;
      float *dst = left    ? part + ((size_t)c * 2) * D
                   : right ? part + ((size_t)c * 2 + 1) * D
                           : dtable + (size_t)k * D;
      const float m = left || right ? 1.f : scale;
      if (v < nv)
#pragma unroll
        for (int j = 0; j < N; j += 4)
          *(float4 *)(dst + (size_t)v * N + j) =
              make_float4(acc[j] * m, acc[j + 1] * m, acc[j + 2] * m, acc[j + 3] * m);
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = 0.f;
      left = false;
    }
  }
}

// ---- step 3: runs that cross chunk ends ----------------------------------------
// A run that begins in chunk c and goes on into chunk c + 1 has the parts
// [c][1] and [c+1][0], [c+2][0], ... up to the chunk it ends in.  A CTA looks
// at `per` chunks (up to eight), a warp each, and adds up those runs' parts for
// 256 columns: four groups of 64 threads take consecutive quarters of the parts,
// whose sums are added in order.  Latency bounds it: a chunk's entries, those on
// both sides and 14 more are one load, and where the chunks are few each has a
// CTA (1000 tokens, V 1000, D 256: 2.6 us less than with eight chunks a CTA).
__global__ void __launch_bounds__(256)
embed_join_kernel(const uint32_t *key, int T, int V, int D, int chunks, int per, float scale,
                  const float *part, float *dtable) {
  pdl_begin();
  __shared__ int s_parts[8];  // parts after the first; 0: nothing begins here and goes on
  __shared__ uint32_t s_key[8];
  __shared__ float4 s_sum[4][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < per) {
    const uint32_t NONE = 0xFFFFFFFFu;
    const int c = (int)blockIdx.x * per + warp;
    int n = 0;
    uint32_t k = NONE;
    if (c < chunks - 1) {
      // lane 0: the entry before the chunk; 1 .. CHUNK: the chunk; then the next
      static_assert(CHUNK + 2 <= 32, "a warp holds a chunk and its neighbours");
      const int at = c * CHUNK + lane - 1;
      const uint32_t k_of = at >= 0 && at < T ? key[at] : NONE;
      k = __shfl_sync(NONE, k_of, CHUNK);
      const uint32_t same = __ballot_sync(NONE, k_of == k);
      // (sorted: the chunk and the entry before it hold one key where their ends do)
      if (k < (uint32_t)V && (same >> (CHUNK + 1) & 1) && !((same & 1) && (same >> 1 & 1))) {
        // the last entry with this key
        int lo = c * CHUNK + 30 - __clz(same), hi = T;  // key[lo] == k
        if (same >> 31 && lo + 1 < T) {  // 32 probes a step; key[hi] > k (or hi == T)
          while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int probe = lo + lane * step;
            const uint32_t holds = __ballot_sync(NONE, probe < hi && key[probe] == k);
            const int last = 31 - __clz(holds);  // (lane 0 holds)
            hi = min(hi, lo + (last + 1) * step);
            lo = lo + last * step;
          }
        }
        n = lo / CHUNK - c;
      }
    }
    if (lane == 0) {
      s_parts[warp] = n;
      s_key[warp] = k;
    }
  }
  __syncthreads();
  const int g = threadIdx.x >> 6, t = threadIdx.x & 63;
  const int col = (int)blockIdx.y * 256 + t * 4;
  for (int w = 0; w < per; ++w) {
    const int n = s_parts[w], c = (int)blockIdx.x * per + w;
    if (n == 0) continue;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < D) {
      if (g == 0) acc = *(const float4 *)(part + ((size_t)c * 2 + 1) * D + col);
      const int a = (int)((long long)n * g / 4), b = (int)((long long)n * (g + 1) / 4);
#pragma unroll 8
      for (int i = a; i < b; ++i) {
        const float4 p = *(const float4 *)(part + (size_t)(c + 1 + i) * 2 * D + col);
        acc.x += p.x; acc.y += p.y; acc.z += p.z; acc.w += p.w;
      }
    }
    s_sum[g][t] = acc;
    __syncthreads();
    if (g == 0 && col < D) {
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        const float4 p = s_sum[i][t];
        acc.x += p.x; acc.y += p.y; acc.z += p.z; acc.w += p.w;
      }
      *(float4 *)(dtable + (size_t)s_key[w] * D + col) =
          make_float4(acc.x * scale, acc.y * scale, acc.z * scale, acc.w * scale);
    }
    __syncthreads();
  }
}

// ---- few tokens: one launch ------------------------------------------------------
// Up to FEW tokens every CTA reads them all.  A warp per position and 32
// vectors of columns: if no earlier position has its token, it adds up the rows
// of all that have, in order.  The other CTAs each zero a range of table rows
// that no position names.  us, one launch | sort, runs and join: 64 tokens, V
// 512, D 128 fp32 6.5 | 11.0; 512 tokens, V 5001, D 512 8.6 | 17.1; 512 tokens
// of 20, D 2048 14.5 | 13.7 (25 rows to a sum, one warp each: from about there
// on the sort pays).
constexpr int FEW = 512;
constexpr int FEW_ROWS = 2048;  // most table rows of a zeroing CTA

template <typename E, typename I>
__global__ void __launch_bounds__(256)
embed_few_kernel(const I *tokens, const E *dy, int T, int V, int nv, float scale,
                 long long pad_id, int sum_ctas, int rows_per, float *dtable, int32_t *status) {
  pdl_begin();
  constexpr int N = VEC16<E>, U = 8;
  const size_t D = (size_t)nv * N;
  if ((int)blockIdx.x >= sum_ctas) {  // zeros
    __shared__ uint8_t named[FEW_ROWS];
    const int v0 = ((int)blockIdx.x - sum_ctas) * rows_per, v1 = v0 + min(rows_per, V - v0);
    for (int i = threadIdx.x; i < v1 - v0; i += 256) named[i] = 0;
    __syncthreads();
    for (int t = threadIdx.x; t < T; t += 256) {
      const uint32_t k = token_key(tokens, t, V, pad_id, nullptr);
      if (k >= (uint32_t)v0 && k < (uint32_t)v1) named[k - v0] = 1;
    }
    __syncthreads();
    const int q = (int)(D / 4);  // 16-byte vectors of a row
    if (q < 32) {                // short rows: a thread a vector
      uint4 *rows = (uint4 *)(dtable + (size_t)v0 * D);
      for (int i = threadIdx.x; i < (v1 - v0) * q; i += 256)
        if (!named[i / q]) rows[i] = make_uint4(0, 0, 0, 0);
      return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int v = v0 + warp; v < v1; v += 8) {
      if (named[v - v0]) continue;
      uint4 *row = (uint4 *)(dtable + (size_t)v * D);
      for (int i = lane; i < q; i += 32) row[i] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  __shared__ uint32_t key[FEW];
  for (int t = threadIdx.x; t < T; t += 256) key[t] = token_key(tokens, t, V, pad_id, status);
  __syncthreads();
  const int lane = threadIdx.x & 31, parts = (nv + 31) / 32;
  const int unit = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = unit / parts, v = (unit - t * parts) * 32 + lane;
  if (t >= T) return;
  const uint32_t k = key[t];
  if (k >= (uint32_t)V) return;
  bool earlier = false;
  for (int i = lane; i < t; i += 32) earlier |= key[i] == k;
  if (__any_sync(0xFFFFFFFFu, earlier)) return;
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.f;
  for (int i0 = t & ~31; i0 < T; i0 += 32) {
    uint32_t m = __ballot_sync(0xFFFFFFFFu, i0 + lane < T && key[i0 + lane] == k);
    while (m) {  // (earlier positions do not match)
      uint4 r[U];
      int n = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!m) break;
        const int at = i0 + __ffs(m) - 1;
        m &= m - 1;
        r[u] = v < nv ? ldg_stream((const uint4 *)dy + (size_t)at * nv + v) : make_uint4(0, 0, 0, 0);
        n = u + 1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= n) break;
        float f[N];
        unpack(r[u], f, (E *)nullptr);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += f[j];
      }
    }
  }
  if (v >= nv) return;
  float *dst = dtable + (size_t)k * D + (size_t)v * N;
#pragma unroll
  for (int j = 0; j < N; j += 4)
    *(float4 *)(dst + j) = make_float4(acc[j] * scale, acc[j + 1] * scale, acc[j + 2] * scale,
                                       acc[j + 3] * scale);
}

template <typename E, typename I>
cudaError_t embed_forward_t(const EmbedArgs &a, const void *table, void *out, cudaStream_t s) {
  const int nv = (int)((size_t)a.D * sizeof(E) / 16);
  const long long units = (long long)a.T * ((nv + 127) / 128);
  const long long grid = (units + 7) / 8;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return launch_k(embed_forward_kernel<E, I>, dim3((unsigned)grid), dim3(256), 0, s,
                  (const I *)a.tokens, (const E *)table, a.T, a.V, nv, a.scale, a.pad_id, (E *)out,
                  a.status);
}

template <typename E, typename I>
cudaError_t embed_backward_t(const EmbedArgs &a, const void *dy, float *dtable,
                             const EmbedScratch &w, cudaStream_t s) {
  const int nv = (int)((size_t)a.D * sizeof(E) / 16);
  if (a.T <= FEW) {
    const int sum_ctas = (a.T * ((nv + 31) / 32) + 7) / 8;
    long long rows = (32 << 10) / ((long long)a.D * 4);  // 32 KB of zeros a CTA
    rows = rows < 8 ? 8 : rows > FEW_ROWS ? FEW_ROWS : rows;
    const long long grid = sum_ctas + (a.V + rows - 1) / rows;
    const cudaError_t e =
        launch_k(embed_few_kernel<E, I>, dim3((unsigned)grid), dim3(256), 0, s,
                 (const I *)a.tokens, (const E *)dy, a.T, a.V, nv, a.scale, a.pad_id, sum_ctas,
                 (int)rows, dtable, a.status);
    prof_mark(KID_EMBED_RUNS, s);
    return e;
  }
  // keys 0 .. V
  int need = 1;
  while (((long long)1 << need) <= a.V) ++need;
  const int passes = (need + DIGIT_MAX - 1) / DIGIT_MAX;
  const int bits = (need + passes - 1) / passes;
  static const cudaError_t attr = [] {
    const cudaError_t e =
        cudaFuncSetAttribute(embed_sort_zero_kernel<I>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortSmem));
    return e != cudaSuccess
               ? e
               : cudaFuncSetAttribute(embed_alone_zero_kernel<I>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      sizeof(AloneSmem));
  }();
  if (attr != cudaSuccess) return attr;
  const size_t table_vecs = (size_t)a.V * a.D / 4;
  const size_t zero_ctas = (table_vecs + ZERO_VECS - 1) / ZERO_VECS;
  const size_t grid = SORT_CTAS + (zero_ctas + SORT_CTAS - 1) / SORT_CTAS * SORT_CTAS;
  if (grid > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  cudaError_t e =
      a.T <= ALONE && passes <= 2
          ? launch_k(embed_alone_zero_kernel<I>, dim3((unsigned)(zero_ctas + 1)),
                     dim3(SORT_THREADS), sizeof(AloneSmem), s, (const I *)a.tokens, a.T, a.V,
                     a.pad_id, w.key[0], w.pos[0], passes, bits, (uint4 *)dtable, table_vecs,
                     a.status)
          : launch_clusters(embed_sort_zero_kernel<I>, dim3((unsigned)grid), dim3(SORT_THREADS),
                            sizeof(SortSmem), SORT_CTAS, s, (const I *)a.tokens, a.T, a.V,
                            a.pad_id, w.key[0], w.pos[0], w.key[1], w.pos[1], passes, bits,
                            (uint4 *)dtable, table_vecs, a.status);
  if (e != cudaSuccess) return e;
  prof_mark(KID_EMBED_SORT, s);
  const int chunks = (a.T + CHUNK - 1) / CHUNK;
  int tpr = 32;
  while (tpr < nv && tpr < 256) tpr *= 2;
  const int per = 256 / tpr;
  e = launch_k(embed_runs_kernel<E>, dim3((chunks + per - 1) / per, (nv + tpr - 1) / tpr),
               dim3(256), 0, s, (const uint32_t *)w.key[0], (const int32_t *)w.pos[0],
               (const E *)dy, a.T, a.V, nv, tpr, chunks, a.scale, dtable, w.part);
  if (e != cudaSuccess) return e;
  prof_mark(KID_EMBED_RUNS, s);
  if (chunks > 1) {
    const int slabs = (a.D + 255) / 256;
    const long long most = (long long)chunks * slabs / (8 * num_sms());  // eight CTAs an SM
    const int join = most < 1 ? 1 : most > 8 ? 8 : (int)most;
    e = launch_k(embed_join_kernel, dim3((chunks + join - 1) / join, slabs), dim3(256), 0, s,
                 (const uint32_t *)w.key[0], a.T, a.V, a.D, chunks, join, a.scale,
                 (const float *)w.part, dtable);
    prof_mark(KID_EMBED_JOIN, s);
  }
  return e;
}

}  // namespace

EmbedScratch carve_embed(void *base, int T, int V, int D) {
  EmbedScratch w;
  (void)V;
  size_t off = 0;
  auto take = [&](size_t bytes) -> void * {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return base ? (void *)((char *)base + o) : nullptr;
  };
  for (int i = 0; i < 2; ++i) {
    w.key[i] = (uint32_t *)take(4 * (size_t)T);
    w.pos[i] = (int32_t *)take(4 * (size_t)T);
  }
  const size_t chunks = ((size_t)T + CHUNK - 1) / CHUNK;
  w.part = (float *)take(chunks * 2 * (size_t)D * 4);
  w.bytes = off;
  return w;
}

cudaError_t launch_embed_forward(const EmbedArgs &a, const void *table, void *out, cudaStream_t s) {
  if (a.dtype == TWELL_BF16)
    return a.token_bytes == 8 ? embed_forward_t<bf16, long long>(a, table, out, s)
                              : embed_forward_t<bf16, int32_t>(a, table, out, s);
  return a.token_bytes == 8 ? embed_forward_t<float, long long>(a, table, out, s)
                            : embed_forward_t<float, int32_t>(a, table, out, s);
}

cudaError_t launch_embed_backward(const EmbedArgs &a, const void *dy, float *dtable,
                                  const EmbedScratch &w, cudaStream_t s) {
  if (a.dtype == TWELL_BF16)
    return a.token_bytes == 8 ? embed_backward_t<bf16, long long>(a, dy, dtable, w, s)
                              : embed_backward_t<bf16, int32_t>(a, dy, dtable, w, s);
  return a.token_bytes == 8 ? embed_backward_t<float, long long>(a, dy, dtable, w, s)
                            : embed_backward_t<float, int32_t>(a, dy, dtable, w, s);
}

}  // namespace twell
