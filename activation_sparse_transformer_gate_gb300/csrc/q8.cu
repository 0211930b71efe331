// q8.cu -- product of 8-bit rows: y[m][n] = sa[m] sw[n] sum_k a[m][k] w[n][k]
// (+ bias[n]).
//
// sm_103a has no fast 8-bit integer tensor path, but an 8-bit integer is
// exact in fp16, its products are exact in fp32, and so is their sum while
// it stays below 2^24: the fp16 tensor cores do this product at full speed.
// The operands stay 8-bit in memory and are widened on the SM.
//
// By the rows of a (matmul_t has the rule and the measurements):
//   a decoded row or four   q8_rows_kernel: dp4a, exact int32 sums
//   a batch of them, small  q8_frag_kernel: the weights are widened in
//   weights                 registers and used up there (m16n8k16)
//   up to 128               q8_few_kernel: TMA brings 8-bit weights, warps
//                           widen them into TMEM, where they are the M side
//                           of tcgen05.mma; clusters share k
//   more                    q8_mma_kernel: warps widen the weights into shared
//                           memory, pairs of CTAs (cta_group::2) multiply
// The rows kernel is bound by the weights' bytes, fragments by the widening of a
// in every warp, few by its MMAs' reading of the weights from TMEM and by its start
// (by the weights' bytes where all SMs have several tiles), the pairs by the tensor
// cores: 8192 x 14336 x 4096 in 0.61 to 0.63 ms, 1.55 PFLOP/s under the power limit
// with the launch that widens a.
#include <cuda_fp16.h>
#include <string.h>

#include "common.cuh"
#include "lm_kernels.h"
#include "tcgen05.cuh"
#include "test_hooks.h"
#include "vec16.cuh"

namespace twell {

namespace {

// ---- few rows ----------------------------------------------------------------
constexpr int ROWS_MAX = 4;  // rows of a that q8_rows_kernel takes
constexpr int ROWS_N = 4;    // weight rows a warp reads together

// A group of KS warps takes ROWS_N weight rows and splits K; MT rows of a
// (M <= MT) are read again by every warp, from L1.  Sums are integers, so
// the split leaves no trace.  Loads in flight bound it: four CTAs an SM and two
// steps ahead for one or two rows, two and four for more (1 x 14336 x 4096 11.8
// us, and 13.4 where the compiler took fewer registers; 4 x 14336 x 16384 42 us,
// three CTAs and two steps 54).
template <typename E, int MT>
__global__ void __launch_bounds__(256, MT <= 2 ? 4 : 2)
q8_rows_kernel(const int8_t *a, const int8_t *w, const float *sa, const float *sw,
               const float *bias, int M, int N, int K, int ks, E *y) {
  pdl_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = ((int)blockIdx.x * (8 / ks) + warp / ks) * ROWS_N;
  const int part = warp % ks;
  const int nv = K / 16;
  int acc[ROWS_N][MT];
#pragma unroll
  for (int r = 0; r < ROWS_N; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = 0;
  if (n0 < N) {
    const uint4 *wr[ROWS_N];
#pragma unroll
    for (int r = 0; r < ROWS_N; ++r)
      wr[r] = (const uint4 *)w + (size_t)min(n0 + r, N - 1) * nv;
    constexpr int STEPS = MT <= 2 ? 2 : 4;
#pragma unroll STEPS
    for (int v = part * 32 + lane; v < nv; v += ks * 32) {
      uint4 x[ROWS_N];
#pragma unroll
      for (int r = 0; r < ROWS_N; ++r) x[r] = ldg_stream(wr[r] + v);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint4 t = __ldg((const uint4 *)a + (size_t)min(m, M - 1) * nv + v);
#pragma unroll
        for (int r = 0; r < ROWS_N; ++r) {
          int s = acc[r][m];
          s = __dp4a((int)x[r].x, (int)t.x, s);
          s = __dp4a((int)x[r].y, (int)t.y, s);
          s = __dp4a((int)x[r].z, (int)t.z, s);
          acc[r][m] = __dp4a((int)x[r].w, (int)t.w, s);
        }
      }
    }
  }
  __shared__ int sums[8][ROWS_N * MT];
#pragma unroll
  for (int r = 0; r < ROWS_N; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int s = __reduce_add_sync(0xFFFFFFFFu, acc[r][m]);
      if (lane == 0) sums[warp][r * MT + m] = s;
    }
  if (ks > 1) __syncthreads();
  else __syncwarp();
  if (part != 0 || lane >= ROWS_N * MT || n0 >= N) return;
  int s = 0;
  for (int i = 0; i < ks; ++i) s += sums[warp + i][lane];
  const int n = n0 + lane / MT, m = lane % MT;
  if (n < N && m < M)
    y[(size_t)m * N + n] = from_f<E>((float)s * sa[m] * sw[n] + (bias ? bias[n] : 0.f));
}

// 16 8-bit integers as fp16: b + 128 under the exponent of 1024 is the fp16
// number 1152 + b.  A word's bytes come out in the order 0, 2, 1, 3: the sum
// over k does not mind, as both operands take the same order.
__device__ __forceinline__ void widen16(const uint4 &v, uint4 &lo, uint4 &hi) {
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[8];
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = (in[i] & 0x00FF00FFu) ^ 0x64806480u;
    const uint32_t q = ((in[i] >> 8) & 0x00FF00FFu) ^ 0x64806480u;
    const __half2 hp = __hsub2(*(const __half2 *)&p, off), hq = __hsub2(*(const __half2 *)&q, off);
    out[2 * i] = *(const uint32_t *)&hp;
    out[2 * i + 1] = *(const uint32_t *)&hq;
  }
  lo = make_uint4(out[0], out[1], out[2], out[3]);
  hi = make_uint4(out[4], out[5], out[6], out[7]);
}

// ---- a batch of decoded rows ---------------------------------------------------
// The weights still stream once from HBM and are used up in registers: a
// warp takes MT times 16 weight rows as the M side of m16n8k16 and NT groups
// of eight rows of a as its N side.  A lane loads 16 consecutive bytes of a
// row, which serve as its part of four MMAs' k (both operands take the same
// order of k), and widens them in registers: rows of a again in every warp,
// which is what bounds it from 32 rows on (reading them widened instead, from
// L1, was slower: 47 against 33 us at 16 x 50001 x 2048, a size that few has now).  A tile's KS warps
// split K and are added in order through shared memory.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The fp16 words of 16 8-bit integers in the order that widen16 gives them.
__device__ __forceinline__ void widen_words(const uint4 &v, uint32_t (&o)[8]) {
  uint4 lo, hi;
  widen16(v, lo, hi);
  o[0] = lo.x; o[1] = lo.y; o[2] = lo.z; o[3] = lo.w;
  o[4] = hi.x; o[5] = hi.y; o[6] = hi.z; o[7] = hi.w;
}

template <typename E, int NT, int MT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 2)
q8_frag_kernel(const uint4 *a, const int8_t *w, const float *sa, const float *sw,
               const float *bias, int M, int N, int K, int ks, E *y) {
  pdl_begin();
  constexpr int ROWS = MT * 16, U = 2;
  __shared__ float sums[WARPS][NT * 8][ROWS + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int tile = (int)blockIdx.x * (WARPS / ks) + warp / ks, part = warp % ks;
  const int n0 = tile * ROWS;
  const int chunks = (K + 63) / 64;
  float acc[MT][NT][4];
#pragma unroll
  for (int h = 0; h < MT; ++h)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[h][j][i] = 0.f;
  if (n0 < N) {
    const int8_t *row[2 * MT];
#pragma unroll
    for (int h = 0; h < 2 * MT; ++h) row[h] = w + (size_t)min(n0 + g + 8 * h, N - 1) * K;
    for (int c = part; c < chunks; c += U * ks) {
      uint4 x[U][2 * MT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (c + u * ks) * 64 + t * 16;
#pragma unroll
        for (int h = 0; h < 2 * MT; ++h)
          x[u][h] = k < K ? ldg_stream(row[h] + k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (c + u * ks) * 64 + t * 16;
        uint32_t p[2 * MT][8];
#pragma unroll
        for (int h = 0; h < 2 * MT; ++h) widen_words(x[u][h], p[h]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const size_t at = ((size_t)min(j * 8 + g, M - 1) * K + k) / 16;
          uint32_t r[8];
          widen_words(k < K ? __ldg(a + at) : make_uint4(0, 0, 0, 0), r);
#pragma unroll
          for (int h = 0; h < MT; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_16816(acc[h][j], p[2 * h][2 * i], p[2 * h + 1][2 * i], p[2 * h][2 * i + 1],
                        p[2 * h + 1][2 * i + 1], r[2 * i], r[2 * i + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < MT; ++h)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sums[warp][j * 8 + 2 * t + (i & 1)][h * 16 + g + (i >> 1) * 8] = acc[h][j][i];
  __syncthreads();
  // the CTA's tiles: `cols` columns of y for each row of a
  const int cols = WARPS / ks * ROWS;
  for (int i = threadIdx.x; i < M * cols; i += WARPS * 32) {
    const int m = i / cols, c = i - m * cols, n = (int)blockIdx.x * cols + c;
    if (n >= N) continue;
    float s = 0.f;
    for (int r = 0; r < ks; ++r) s += sums[c / ROWS * ks + r][m][c % ROWS];
    y[(size_t)m * N + n] = from_f<E>(s * sa[m] * sw[n] + (bias ? bias[n] : 0.f));
  }
}

// ---- tensor cores --------------------------------------------------------------
constexpr int BM = 128, BK = 64;
constexpr int ACC_COLS = 256;  // TMEM columns of one accumulator
constexpr int GROUPS = 4;      // conversion groups, which take the k-blocks in turn

// A pair of CTAs per tile: rows of a; stages of a (fp16), of w in fp16 and in 8
// bits, with 128 rows each; warps of a conversion group.
constexpr int ROWS = 2 * BM;
constexpr int AS = 5, WS = 4, RS = 8;
constexpr int GROUP = 2;
constexpr int THREADS = 32 * (8 + GROUPS * GROUP);
constexpr int TILE = BM * BK * 2, RAW = BM * BK;  // bytes of a stage
constexpr int SMEM = 1024 + (AS + WS) * TILE + RS * RAW + 2 * 256 * 4;

struct Q8Maps {
  CUtensorMap a, w;
};

struct Q8Params {
  int M, N, K;
  int bn;   // output columns of a tile
  const float *sa, *sw, *bias;
  void *y;
  int32_t *status;
};

__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void scale32(float *v, float sa, const float *sw, const float *bias) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 s = *(const float4 *)(sw + i), b = *(const float4 *)(bias + i);
    v[i] = v[i] * sa * s.x + b.x;
    v[i + 1] = v[i + 1] * sa * s.y + b.y;
    v[i + 2] = v[i + 2] * sa * s.z + b.z;
    v[i + 3] = v[i + 3] * sa * s.w + b.w;
  }
}

// 32 values of a row, rounded, as the words behind e[0 .. 3].
__device__ __forceinline__ void row_words(const float (&v)[32], uint32_t (&e)[36], float *) {
#pragma unroll
  for (int i = 0; i < 32; ++i) e[4 + i] = __float_as_uint(v[i]);
}
__device__ __forceinline__ void row_words(const float (&v)[32], uint32_t (&e)[20], bf16 *) {
#pragma unroll
  for (int i = 0; i < 16; ++i) e[4 + i] = pack_bf2(v[2 * i], v[2 * i + 1]);
}
// e[4 ..] becomes what stands r elements before it.
__device__ __forceinline__ void move_words(uint32_t (&e)[36], int r, float *) {
  const bool r1 = r & 1, r2 = r & 2;
#pragma unroll
  for (int i = 35; i >= 1; --i) e[i] = r1 ? e[i - 1] : e[i];
#pragma unroll
  for (int i = 35; i >= 4; --i) e[i] = r2 ? e[i - 2] : e[i];
}
__device__ __forceinline__ void move_words(uint32_t (&e)[20], int r, bf16 *) {
  const uint32_t r1 = r & 1 ? 0x5432 : 0x7654;
  const bool r2 = r & 2, r4 = r & 4;
#pragma unroll
  for (int i = 19; i >= 1; --i) e[i] = __byte_perm(e[i - 1], e[i], r1);
#pragma unroll
  for (int i = 19; i >= 2; --i) e[i] = r2 ? e[i - 1] : e[i];
#pragma unroll
  for (int i = 19; i >= 4; --i) e[i] = r4 ? e[i - 2] : e[i];
}
// Elements lo <= j < hi of a vector.
__device__ __forceinline__ void store_some(float *dst, const uint32_t *w, int lo, int hi) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j >= lo && j < hi) dst[j] = __uint_as_float(w[j]);
}
__device__ __forceinline__ void store_some(bf16 *dst, const uint32_t *w, int lo, int hi) {
  // from lo up to what is aligned to 2, 4, 8 elements, and from there down to hi
  auto word = [&](int i) { return i & 2 ? i & 1 ? w[3] : w[2] : i & 1 ? w[1] : w[0]; };
  if ((lo & 1) && lo < hi) {
    ((uint16_t *)dst)[lo] = (uint16_t)(word(lo >> 1) >> 16);
    ++lo;
  }
  if ((lo & 2) && lo + 2 <= hi) {
    *(uint32_t *)(dst + lo) = word(lo >> 1);
    lo += 2;
  }
  if (lo + 4 <= hi) {
    *(uint2 *)(dst + lo) = lo ? make_uint2(w[2], w[3]) : make_uint2(w[0], w[1]);
    lo += 4;
  }
  if (lo + 2 <= hi) {
    *(uint32_t *)(dst + lo) = word(lo >> 1);
    lo += 2;
  }
  if (lo < hi) ((uint16_t *)dst)[lo] = (uint16_t)word(lo >> 1);
}

// One warp's 32 accumulator rows (TMEM lane = row, from row m0 on) of a tile of
// bn columns from n0 on: scaled, rounded, and stored by each thread for its own
// row, in 16 bytes at a time whatever the row's alignment: its elements move by
// as many places as the row starts behind a 16-byte boundary, and the first and
// the last few are stored alone, in the widest pieces.  (Stores count by
// their number: 1001 x 50001 x 512, where rows of y start at odd elements and
// the epilogue is all there is, takes 71 us, with 50000 columns 65; through
// shared memory, in words that a warp stores for one row, it took 118, and 1001
// x 50001 x 2048 151 us instead of 144.)
template <typename E>
__device__ __forceinline__ void store_tile(const Q8Params &p, E *y, uint32_t acc, int m0, int n0,
                                           float sa, const float *s_sw) {
  constexpr int N = VEC16<E>, WORDS = 32 * (int)sizeof(E) / 4;  // of 32 columns
  const int lane = threadIdx.x & 31, cols = min(p.bn, p.N - n0);
  E *row = y + (size_t)(m0 + lane) * p.N + n0;
  const int r = (int)((uintptr_t)row / sizeof(E)) & (N - 1);
  row -= r;
  const int end = m0 + lane < p.M ? r + cols : 0;
  // the vector from element `at` on
  auto store = [&](const uint32_t *w, int at) {
    const int lo = at == 0 ? r : 0, hi = end - at;
    if (lo == 0 && hi >= N)
      *(uint4 *)(row + at) = make_uint4(w[0], w[1], w[2], w[3]);
    else if (hi > lo)
      store_some(row + at, w, lo, hi);
  };
  uint32_t e[4 + WORDS], last[4] = {};
  int c0 = 0;
  for (; c0 < cols; c0 += 32) {
    float v[32];
    __syncwarp();  // (tcgen05.ld takes the whole warp)
    tmem_ld32(acc + c0, v);
    scale32(v, sa, s_sw + c0, s_sw + 256 + c0);
    row_words(v, e, (E *)nullptr);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[i] = last[i];
      last[i] = e[WORDS + i];
    }
    move_words(e, r, (E *)nullptr);
#pragma unroll
    for (int j = 0; j < 32; j += N) store(e + 4 + j * (int)sizeof(E) / 4, c0 + j);
  }
  // what has moved past the last 32 columns
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = last[i];
    e[4 + i] = 0;
  }
  move_words(e, r, (E *)nullptr);
  store(e + 4, c0);
}

// Scale and bias of a tile's columns, staged by the 128 epilogue threads.
__device__ __forceinline__ void stage_columns(const Q8Params &p, int n0, float *s_sw, int et) {
  epi_bar();
  for (int c = et; c < p.bn; c += 128) {
    s_sw[c] = n0 + c < p.N ? p.sw[n0 + c] : 0.f;
    s_sw[256 + c] = p.bias && n0 + c < p.N ? p.bias[n0 + c] : 0.f;
  }
  epi_bar();
}

// One k-block's conversion by CT threads: the `vecs` 16-byte vectors (a
// multiple of 32) of rows of 64 8-bit values at src become fp16 rows of 128
// bytes (128B swizzle) at dst.  Thread ct takes vectors ct, ct + CT, ...: the
// same place in every (CT / 4)th row, so the addresses differ by constants.
template <int CT>
__device__ __forceinline__ void widen_rows(const uint8_t *src, uint8_t *dst, int ct, int vecs) {
  static_assert(CT % 32 == 0, "the swizzle phase of a thread's rows is one");
  constexpr int B = 4;  // vectors in flight
  const int r = ct >> 2, c = (ct & 3) * 2;
  uint8_t *row = dst + r * 128;
  uint4 *lo = (uint4 *)(row + ((c ^ (r & 7)) * 16)), *hi = (uint4 *)(row + (((c + 1) ^ (r & 7)) * 16));
  const uint4 *p = (const uint4 *)src + ct;
  for (int v = ct; v < vecs; v += B * CT) {
    uint4 x[B];
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (v + i * CT < vecs) x[i] = p[i * CT];
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (v + i * CT < vecs) widen16(x[i], lo[i * (CT * 2)], hi[i * (CT * 2)]);
    p += B * CT;
    lo += B * CT * 2;
    hi += B * CT * 2;
  }
}

// Stage and phase of a ring of S stages, for a user of every STEP-th stage.
struct Ring {
  int at;
  uint32_t phase;
  __device__ __forceinline__ Ring(int first, int S) : at(first % S), phase((first / S) & 1) {}
  template <int STEP = 1>
  __device__ __forceinline__ void next(int S) {
    at += STEP;
    while (at >= S) {
      at -= S;
      phase ^= 1;
    }
  }
};

// A wait that a whole warp takes together: all lanes go on or all give up, so
// that the warp stays whole for what follows.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                          int32_t *status) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, status));
}

// No copy may be in flight when the CTA exits: waits (bounded) for the last
// load that was issued into each stage of a ring.  That the issuing warp has
// come to its end does not say that the loads were waited for: another role may
// have given up since.  (So for commits, where `full` are the barriers at which
// they arrive.)
__device__ __forceinline__ void drain_ring(uint32_t full, int S, long issued) {
  for (int s = 0; s < S && s < issued; ++s) {
    const uint32_t par = (uint32_t)(((issued - 1 - s) / S) & 1);
    const uint64_t t0 = global_timer();
    while (!mbar_try(full + 8 * s, par) && global_timer() - t0 < DRAIN_LIMIT_NS) {
    }
  }
}

#ifdef TWELL_TEST_HOOKS
// CTAs of pairs that have ended, and those among them that left while an
// arrival at one of their barriers was still to come.
__device__ unsigned test_pairs[2];
__device__ __forceinline__ bool ring_drained(uint32_t full, int S, long issued) {
  for (int s = 0; s < S && s < issued; ++s)
    if (!mbar_test(full + 8 * s, (uint32_t)(((issued - 1 - s) / S) & 1))) return false;
  return true;
}
#endif

// Address part of the swizzled operand descriptors (sw128_desc): adding to
// the low word moves the start, 16 bytes a unit.
__device__ __forceinline__ uint64_t desc_at(uint32_t saddr) { return sw128_desc(saddr, 16, 1024); }

// ---- more than 128 rows of a ---------------------------------------------------
// a is widened once by q8_widen_kernel and comes by TMA as fp16; w comes by
// TMA in 8 bits and is widened here, between two stages of shared memory.
//
// Two CTAs (one cluster) share a 256 x bn tile: each holds 128 rows of a and bn
// / 2 rows of w, the leader issues cta_group::2 MMAs over both, and each CTA
// stores its 128 rows.  Per k-block an SM then moves 64 KB through shared memory
// (w in 8 bits twice and in fp16 once, a once, the MMA's reads) where one CTA
// that widened both operands for its own 128 x 256 tile would move 144 KB for
// the same multiplications, and shared memory, not the tensor cores, was its
// bound (770 TFLOP/s at M 8192, N 14336, K 4096; pairs: 1.7 PFLOP/s).
//
// A conversion warp's loads, stores, their fence and its arrival take about
// 2000 cycles from end to end, four times a k-block's MMAs, so four groups of
// warps take the k-blocks in turn.  They arrive at a barrier of their own CTA
// and one thread passes that on to the leader.

// fp16 copy of a.
__global__ void __launch_bounds__(256)
q8_widen_kernel(const uint4 *a, size_t vecs, uint4 *out) {
  pdl_begin();
  pdl_trigger();  // (the product's weights are under way meanwhile)
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= vecs) return;
  uint4 lo, hi;
  widen16(ldg_stream<L2_FIRST>(a + i), lo, hi);
  out[2 * i] = lo;
  out[2 * i + 1] = hi;
}

template <typename E>
__global__ void __launch_bounds__(THREADS, 1)
q8_mma_kernel(const __grid_constant__ Q8Maps maps, const __grid_constant__ Q8Params p) {
  // (everything but the fp16 rows of a was complete before q8_widen_kernel:
  // only their producer waits for it)
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sa16 = smem, *sw16 = sa16 + AS * TILE, *raw = sw16 + WS * TILE;
  float *s_sw = (float *)(raw + RS * RAW);
  // Barriers of this CTA: a stage is full, a stage is free again.  Barriers of
  // the leader, at which both CTAs arrive: a k-block's operands are ready, an
  // accumulator has been read (tempty).
  __shared__ uint64_t bars[2 * AS + 3 * WS + 2 * RS + 5];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ uint32_t s_committed[2];  // k-blocks and tiles that the leader has committed
  volatile int *abort_flag = &s_abort;
  const uint32_t afull = smem_u32(bars), aempty = afull + 8 * AS;
  const uint32_t wfull = aempty + 8 * AS, wempty = wfull + 8 * WS, ready = wempty + 8 * WS;
  const uint32_t rfull = ready + 8 * WS, rempty = rfull + 8 * RS;
  const uint32_t tfull = rempty + 8 * RS, tempty = tfull + 16, mma_done = tempty + 16;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x & 1);  // (a pair's CTAs are consecutive)
  const int bn = p.bn, half = bn / 2;      // columns of the tile; rows of w here

  const int mb = (p.M + ROWS - 1) / ROWS, nb = (p.N + bn - 1) / bn;
  const int tiles = mb * nb;  // M-blocks innermost: the tiles in flight share few weight tiles
  const int KT = (p.K + BK - 1) / BK;
  // this pair's tiles: unit, unit + units, ...; their k-blocks
  const int unit = (int)blockIdx.x >> 1, units = (int)gridDim.x >> 1;
  const long its = (long)((tiles - unit + units - 1) / units) * KT;

  if (threadIdx.x == 0) {
    for (int i = 0; i < AS; ++i) {
      mbar_init(afull + 8 * i, 1);
      mbar_init(aempty + 8 * i, 1);
    }
    for (int i = 0; i < WS; ++i) {
      mbar_init(wfull + 8 * i, GROUP);
      mbar_init(wempty + 8 * i, 1);
      mbar_init(ready + 8 * i, 2);
    }
    for (int i = 0; i < RS; ++i) {
      mbar_init(rfull + 8 * i, 1);
      mbar_init(rempty + 8 * i, GROUP);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, 8);
    }
    mbar_init(mma_done, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<true>(smem_u32(&s_tmem), 2 * ACC_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == 0 || warp == 6) {
    // ------------------------------- TMA producers: w in 8 bits; a in fp16 --
    const bool issues = elect_one();
    const bool is_w = warp == 0;
    if (!is_w) pdl_begin();
    const uint32_t full = is_w ? rfull : afull, empty = is_w ? rempty : aempty;
    const uint32_t dst0 = smem_u32(is_w ? raw : sa16), step = is_w ? RAW : TILE;
    const int stages = is_w ? RS : AS, bytes = is_w ? half * BK : BM * BK * 2;
    const CUtensorMap *map = is_w ? &maps.w : &maps.a;
    int st = 0;
    uint32_t ph = 0;
    long issued = 0;
    bool ok = true;
    for (int t = unit; t < tiles && ok; t += units) {
      const int row = is_w ? (t / mb) * bn + rank * half : (t % mb) * ROWS + rank * BM;
      for (int kt = 0; kt < KT; ++kt) {
        ok = warp_wait(empty + 8 * st, ph ^ 1, abort_flag, p.status);
        if (!ok) break;
        if (issues) {
          mbar_expect_tx(full + 8 * st, (uint32_t)bytes);
          tma_load_2d(dst0 + st * step, map, kt * BK, row, full + 8 * st);
        }
        __syncwarp();
        ++issued;
        if (++st == stages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    drain_ring(full, stages, issued);
  } else if (warp == 7) {
    // ------------- tells the leader that this CTA's operands have arrived --
    if (lane == 0) {
      const uint32_t to = cluster_addr(ready, 0);
      Ring a(0, AS), w(0, WS);
      for (long it = 0; it < its; ++it) {
        if (!mbar_wait(afull + 8 * a.at, a.phase, abort_flag, p.status) ||
            !mbar_wait(wfull + 8 * w.at, w.phase, abort_flag, p.status))
          break;
        mbar_arrive_cluster(to + 8 * w.at);
        a.next(AS);
        w.next(WS);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer --
    if (rank == 0) {
      const bool issues = elect_one();
      const uint32_t idesc = make_idesc(ROWS, bn, false, false, true);
      const uint64_t ad0 = desc_at(smem_u32(sa16)), wd0 = desc_at(smem_u32(sw16));
      Ring a(0, AS), w(0, WS);
      int lt = 0;
      bool ok = true;
      int seen = 0;
      uint32_t blocks = 0, done = 0;  // committed k-blocks, tiles
      for (int t = unit; t < tiles && ok; t += units, ++lt) {
        const int buf = lt & 1;
        ok = warp_wait(tempty + 8 * buf, ((uint32_t)(lt >> 1) & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * ACC_COLS);
        for (int kt = 0; kt < KT; ++kt) {
          if (!__all_sync(0xFFFFFFFFu, seen)) {
            ok = warp_wait(ready + 8 * w.at, w.phase, abort_flag, p.status);
            if (!ok) break;
          }
          tc_fence_after();
          const uint64_t ad = ad0 + (uint32_t)(a.at * (TILE >> 4));
          const uint64_t wd = wd0 + (uint32_t)(w.at * (TILE >> 4));
          const uint32_t a_free = aempty + 8 * a.at, w_free = wempty + 8 * w.at;
          a.next(AS);
          w.next(WS);
          seen = mbar_test(ready + 8 * w.at, w.phase);  // of the next one, under this one's issue
          if (issues) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_f16_pair(acc, ad + 2 * kk, wd + 2 * kk, idesc, (kt > 0 || kk > 0) ? 1u : 0u);
            mma_commit_pair(a_free);
            mma_commit_pair(w_free);
          }
          ++blocks;
          __syncwarp();
        }
        if (!ok) break;
        if (issues) mma_commit_pair(tfull + 8 * buf);
        ++done;
        __syncwarp();
      }
      if (issues) mma_commit_pair(mma_done);
      if (lane < 2) {  // (read behind the cluster's barrier)
        st_cluster(cluster_addr(smem_u32(s_committed), lane), blocks);
        st_cluster(cluster_addr(smem_u32(s_committed + 1), lane), done);
      }
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue --
    const int q = warp & 3;  // TMEM lane quadrant of this warp
    const uint32_t free = cluster_addr(tempty, 0);
    int lt = 0;
    for (int t = unit; t < tiles; t += units, ++lt) {
      const int m0 = (t % mb) * ROWS + rank * BM + q * 32, n0 = (t / mb) * bn;
      const int buf = lt & 1;
      stage_columns(p, n0, s_sw, threadIdx.x - 64);
      const float sa = m0 + lane < p.M ? p.sa[m0 + lane] : 0.f;
      const bool ok = epi_all(mbar_wait(tfull + 8 * buf, (uint32_t)(lt >> 1) & 1,
                                                abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
      if (m0 < p.M)  // (uniform for the warp)
        store_tile(p, (E *)p.y, tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * ACC_COLS), m0,
                   n0, sa, s_sw);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(free + 8 * buf);
    }
  } else {
    // ---------------------------------------------------------- conversion --
    const int group = (warp - 8) / GROUP, ct = (threadIdx.x - 256) % (32 * GROUP);
    const int vecs = half * (BK / 16);
    Ring w(group, WS), r(group, RS);
    for (long it = group; it < its; it += GROUPS) {
      // w's stage first: when it is free, the k-blocks up to it - GROUPS have been
      // multiplied, so the 8-bit stage's last load before this one (it - RS, of
      // another group) has been seen and the phase's parity means this one
      if (!warp_wait(wempty + 8 * w.at, w.phase ^ 1, abort_flag, p.status)) break;
      if (!warp_wait(rfull + 8 * r.at, r.phase, abort_flag, p.status)) break;
      widen_rows<32 * GROUP>(raw + r.at * RAW, sw16 + w.at * TILE, ct, vecs);
      fence_async_proxy();  // the MMA reads through the async proxy
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(wfull + 8 * w.at);
        mbar_arrive(rempty + 8 * r.at);
      }
      w.next<GROUPS>(WS);
      r.next<GROUPS>(RS);
    }
  }

  // Neither CTA of a pair leaves while something may still reach its shared
  // memory or TMEM.  The other's threads: the barrier.  The leader's MMAs, which
  // read both CTAs, and its commits, which arrive in both: each CTA waits
  // (bounded) for the last arrival at each of its own barriers that take commits,
  // also where roles have given up, which is why their number is passed on.
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    const long blocks = s_committed[0], done = s_committed[1];
    drain_ring(mma_done, 1, 1);
    drain_ring(aempty, AS, blocks);
    drain_ring(wempty, WS, blocks);
    drain_ring(tfull, 2, done);
#ifdef TWELL_TEST_HOOKS
    if (lane == 0 && (!ring_drained(mma_done, 1, 1) || !ring_drained(aempty, AS, blocks) ||
                      !ring_drained(wempty, WS, blocks) || !ring_drained(tfull, 2, done)))
      atomicAdd(&test_pairs[1], 1u);
    if (lane == 0) atomicAdd(&test_pairs[0], 1u);
#endif
    tc_fence_after();
    tmem_free<true>(tmem, 2 * ACC_COLS);
  }
}

// ---- up to 128 rows of a ------------------------------------------------------
// The product is turned round: 128 rows of w are the M side of tcgen05.mma and
// the rows of a its N side, so an MMA is as wide as there are rows.  w is read
// from TMEM, into which the conversion warps write it as they widen it: in
// shared memory it is only ever in 8 bits.  With w widened there too, and 128
// rows of a read for however few there are, a k-block of 64 for 96 columns moved
// 57 KB through shared memory, which at its 128 bytes a cycle took the 420 cycles
// that were measured (37 x 14336 x 4096: 20.2 us); here 128 k of 128 columns move
// 52 KB and take 600 (16.3 us).
//
// A tile is 128 columns of y.  Where the tiles leave SMs idle, a cluster of ks
// CTAs shares a tile's k and adds the parts through distributed shared memory,
// each CTA for its share of the rows of a (100 x 2048 x 2048: 11.5 us).
//
// What is left above the weights' bytes: an MMA takes 75 cycles however few rows
// of a there are (128 x 16 of w come from TMEM at about 64 bytes a cycle), 600
// a k-block, so 112 tiles keep 112 of 152 SMs below HBM's rate (narrower tiles on
// more SMs take the same time: their MMAs are as high); some 9000 cycles from
// the first load to the first MMA, when all SMs fill their rings at once; 2000
// of the epilogue.  Its stores count by their number: 32 of 64 bytes a warp took
// 4200 cycles for 37 rows, the same bytes in stores of 16 a lane 2100.
constexpr int FEW_MOST = 128;              // rows of a
constexpr int FN = 128, FK = 128;          // columns of y a tile, k of a k-block
constexpr int FEW_STAGES = 6;              // of w in TMEM and of a in shared memory: the most
constexpr int FEW_RAW = 12;                // of w in 8 bits: the most
constexpr int FEW_RINGS = 4 * FEW_MOST * FK * 2 + 6 * FN * FK;
constexpr int FEW_SMEM = 1024 + FEW_RINGS;
constexpr int FEW_THREADS = 32 * (8 + 4 * GROUPS);
constexpr int FEW_BARS = 3 * FEW_STAGES + 2 * FEW_RAW + 5;

struct FewParams {
  int M, N, K;
  int box;         // rows of a that a TMA box holds
  int ks;          // CTAs that share a tile
  int cols;        // rows of a in MMAs: TMEM columns of an accumulator
  int stages, raw_stages;
  const float *sa, *sw, *bias;
  void *y;
  int32_t *status;
};

// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
// The MMA with its first operand in TMEM.
__device__ __forceinline__ void mma_tmem(uint32_t dtmem, uint32_t atmem, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(dtmem),
      "r"(atmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 32 rows of y from row m0 on; this lane holds column n of them (of `rows` rows
// where the column exists).
__device__ __forceinline__ void store_columns(const FewParams &p, float *y, int n, int m0,
                                              int rows, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (m0 + i < rows) y[(size_t)(m0 + i) * p.N] = v[i];
}
__device__ __forceinline__ void store_columns(const FewParams &p, bf16 *y, int n, int m0, int rows,
                                              const float (&v)[32]) {
  if (p.N % 8 != 0) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (m0 + i < rows) y[(size_t)(m0 + i) * p.N] = __float2bfloat16_rn(v[i]);
    return;
  }
  // 8 x 8 blocks change places between eight lanes, which then hold eight
  // columns of one row each
  const int lane = threadIdx.x & 31;
  const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
  uint32_t h[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t own = pack_bf2(v[2 * i], v[2 * i + 1]);
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
    h[i] = b0 ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
  }
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const uint32_t keep = b1 ? h[i + 1] : h[i];
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, b1 ? h[i] : h[i + 1], 2);
    h[i] = b1 ? got : keep;
    h[i + 1] = b1 ? keep : got;
  }
  const int m = m0 + (lane & 7), c = n - lane + (lane >> 3) * 8;
  bf16 *row = (bf16 *)p.y + (size_t)m * p.N + c;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    uint32_t keep[2], got[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      keep[j] = b2 ? h[i + 2 + j] : h[i + j];
      got[j] = __shfl_xor_sync(0xFFFFFFFFu, b2 ? h[i + j] : h[i + 2 + j], 4);
    }
    if (m + 2 * i < p.M && c < p.N)
      *(uint4 *)(row + (size_t)(2 * i) * p.N) =
          b2 ? make_uint4(got[0], got[1], keep[0], keep[1])
             : make_uint4(keep[0], keep[1], got[0], got[1]);
  }
}

template <typename E>
__global__ void __launch_bounds__(FEW_THREADS, 1)
q8_few_kernel(const __grid_constant__ Q8Maps maps, const __grid_constant__ FewParams p) {
  // (everything but the fp16 rows of a was complete before q8_widen_kernel:
  // only their producer waits for it)
  constexpr int RAW = FN * FK;           // bytes of a stage of w in 8 bits
  const int WS = p.stages, RS = p.raw_stages;
  const int half = p.box * 128, a_step = 2 * half;  // bytes: 64 k of a's rows; a stage
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *raw = smem + WS * a_step;  // (behind a: an MMA may read past a stage's rows)
  __shared__ uint64_t bars[FEW_BARS];
  __shared__ __align__(16) float s_sa[FEW_MOST];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;
  const uint32_t afull = smem_u32(bars), wfull = afull + 8 * FEW_STAGES;
  const uint32_t empty = wfull + 8 * FEW_STAGES;  // frees a stage of a and one of w
  const uint32_t rfull = empty + 8 * FEW_STAGES, rempty = rfull + 8 * FEW_RAW;
  const uint32_t tfull = rempty + 8 * FEW_RAW, tempty = tfull + 16, mma_done = tempty + 16;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int tiles = (p.N + FN - 1) / FN, KT = (p.K + FK - 1) / FK;
  // this CTA's tiles: unit, unit + units, ... (one where a tile is shared);
  // its k-blocks of each: [k0, k1)
  const int rank = (int)blockIdx.x % p.ks, unit = (int)blockIdx.x / p.ks;
  const int units = (int)gridDim.x / p.ks;
  const int k0 = (int)((long)KT * rank / p.ks), k1 = (int)((long)KT * (rank + 1) / p.ks);

  // The loads of w begin as soon as their barriers stand: warp 0 only arrives
  // where the others wait for the barriers and for TMEM.
  uint32_t tmem = 0;
  if (warp == 0) {
    for (int i = lane; i < FEW_BARS; i += 32) {
      const uint32_t bar = afull + 8 * i;  // four warps arrive at these, one thread at the others
      const bool four = (bar >= wfull && bar < empty) || (bar >= rempty && bar < tfull) ||
                        (bar >= tempty && bar < mma_done);
      mbar_init(bar, four ? 4 : 1);
    }
    if (lane == 0) s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    asm volatile("bar.arrive 2, %0;" ::"n"(FEW_THREADS) : "memory");
  } else {
    if (warp == 1) tmem_alloc<false>(smem_u32(&s_tmem), 512);
    tc_fence_before();
    asm volatile("bar.sync 2, %0;" ::"n"(FEW_THREADS) : "memory");
    tc_fence_after();
    tmem = s_tmem;
  }
  const uint32_t w16 = tmem + 2 * p.cols;  // behind two accumulators: the stages of w

  if (warp == 0 || warp == 6) {
    // ------------------------------- TMA producers: w in 8 bits; a in fp16 --
    const bool issues = elect_one();
    const bool is_w = warp == 0;
    if (!is_w) pdl_begin();
    const uint32_t full = is_w ? rfull : afull, free = is_w ? rempty : empty;
    const uint32_t dst0 = smem_u32(is_w ? raw : smem), step = is_w ? RAW : a_step;
    const int stages = is_w ? RS : WS;
    Ring r(0, stages);
    long issued = 0;
    bool ok = true;
    for (int t = unit; t < tiles && ok; t += units) {
      for (int kt = k0; kt < k1; ++kt) {
        ok = warp_wait(free + 8 * r.at, r.phase ^ 1, abort_flag, p.status);
        if (!ok) break;
        if (issues) {
          const uint32_t bar = full + 8 * r.at, dst = dst0 + r.at * step;
          mbar_expect_tx(bar, step);
          if (is_w) {
            tma_load_2d(dst, &maps.w, kt * FK, t * FN, bar);
          } else {
            tma_load_2d(dst, &maps.a, kt * FK, 0, bar);
            tma_load_2d(dst + half, &maps.a, kt * FK + 64, 0, bar);
          }
        }
        __syncwarp();
        ++issued;
        r.next(stages);
      }
    }
    drain_ring(full, stages, issued);
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer --
    const bool issues = elect_one();
    const uint32_t idesc = make_idesc(FN, p.cols, false, false, true);
    const uint64_t ad0 = desc_at(smem_u32(smem));
    auto look = [&](const Ring &w) -> int {  // (not one after the other)
      const bool has_w = mbar_test(wfull + 8 * w.at, w.phase);
      const bool has_a = mbar_test(afull + 8 * w.at, w.phase);
      return (int)has_w & (int)has_a;
    };
    Ring w(0, WS);
    int lt = 0, seen = 0;
    bool ok = true;
    for (int t = unit; t < tiles && ok; t += units, ++lt) {
      const int buf = lt & 1;
      ok = warp_wait(tempty + 8 * buf, ((uint32_t)(lt >> 1) & 1) ^ 1, abort_flag, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(buf * p.cols);
      for (int kt = k0; kt < k1; ++kt) {
        if (!__all_sync(0xFFFFFFFFu, seen)) {
          ok = warp_wait(wfull + 8 * w.at, w.phase, abort_flag, p.status) &&
               warp_wait(afull + 8 * w.at, w.phase, abort_flag, p.status);
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t wt = w16 + (uint32_t)(w.at * (FK / 2));
        const uint64_t ad = ad0 + (uint32_t)(w.at * (a_step >> 4));
        const uint32_t done = empty + 8 * w.at;
        w.next(WS);
        seen = look(w);  // of the next k-block, under this one's issue
        __syncwarp();
        if (issues) {
#pragma unroll
          for (int kk = 0; kk < FK / 16; ++kk)
            mma_tmem(acc, wt + 8 * kk, ad + (uint32_t)((kk >> 2) * (half >> 4) + 2 * (kk & 3)),
                     idesc, (kt > k0 || kk > 0) ? 1u : 0u);
          mma_commit(done);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (issues) mma_commit(tfull + 8 * buf);
      __syncwarp();
    }
    // all MMAs issued by this thread are complete before TMEM is freed
    if (issues) mma_commit(mma_done);
    __syncwarp();
    const uint64_t t0 = global_timer();
    while (!mbar_try(mma_done, 0) && global_timer() - t0 < DRAIN_LIMIT_NS) {
    }
  } else if (warp < 6) {
    // ------------------------ epilogue: a lane is a column of y, n0 + lane --
    const int q = warp & 3;  // TMEM lane quadrant of this warp
    float *part = (float *)smem + q * 32 + lane;  // [row of a][FN]; the rings are done with
    const int e = q * 32 + lane;
    s_sa[e] = e < p.M ? p.sa[e] : 0.f;
    epi_bar();
    int lt = 0;
    for (int t = unit; t < tiles; t += units, ++lt) {
      const int n = t * FN + q * 32 + lane, buf = lt & 1;
      const float sw = n < p.N ? p.sw[n] : 0.f, bias = p.bias && n < p.N ? p.bias[n] : 0.f;
      const bool ok = epi_all(mbar_wait(tfull + 8 * buf, (uint32_t)(lt >> 1) & 1, abort_flag,
                                        p.status));
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * p.cols);
      E *y = (E *)p.y + n;
      const int rows = n < p.N ? p.M : 0;
      for (int m0 = 0; m0 < p.M; m0 += 32) {
        float v[32];
        __syncwarp();  // (tcgen05.ld takes the whole warp)
        tmem_ld32(acc + m0, v);
        if (p.ks > 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (m0 + i < p.M) part[(m0 + i) * FN] = v[i];
        } else {
          // (all scales before the first store, behind which they would wait)
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 sa = *(const float4 *)(s_sa + m0 + i);
            v[i] = v[i] * sa.x * sw + bias;
            v[i + 1] = v[i + 1] * sa.y * sw + bias;
            v[i + 2] = v[i + 2] * sa.z * sw + bias;
            v[i + 3] = v[i + 3] * sa.w * sw + bias;
          }
          store_columns(p, y, n, m0, rows, v);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty + 8 * buf);
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------- conversion --
    const int group = (warp - 8) >> 2, row = (warp & 3) * 32 + lane;
    const long its = (long)((tiles - unit + units - 1) / units) * (k1 - k0);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    Ring w(group, WS), r(group, RS);
    for (long it = group; it < its; it += GROUPS) {
      // w's stage first: when it is free, the k-blocks up to it - WS have been
      // multiplied, so the 8-bit stage's last load before this one (it - RS, of
      // another group) has been seen and the phase's parity means this one (so
      // it does for w's stage: MMAs complete in order, and this group has seen
      // those up to it - 4 - WS)
      if (!warp_wait(empty + 8 * w.at, w.phase ^ 1, abort_flag, p.status)) break;
      if (!warp_wait(rfull + 8 * r.at, r.phase, abort_flag, p.status)) break;
      __syncwarp();  // (tcgen05.st takes the whole warp)
      tc_fence_after();
      const uint8_t *src = raw + r.at * RAW + row * FK;  // (128B swizzle)
      const uint32_t dst = w16 + lanes + (uint32_t)(w.at * (FK / 2));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = *(const uint4 *)(src + (((h * 4 + j) ^ (row & 7)) * 16));
        uint32_t f[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 lo, hi;
          widen16(x[j], lo, hi);
          f[8 * j] = lo.x; f[8 * j + 1] = lo.y; f[8 * j + 2] = lo.z; f[8 * j + 3] = lo.w;
          f[8 * j + 4] = hi.x; f[8 * j + 5] = hi.y; f[8 * j + 6] = hi.z; f[8 * j + 7] = hi.w;
        }
        tmem_st32(dst + h * 32, f);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(wfull + 8 * w.at);
        mbar_arrive(rempty + 8 * r.at);
      }
      w.next<GROUPS>(WS);
      r.next<GROUPS>(RS);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free<false>(tmem, 512);
  }
  if (p.ks == 1) return;
  // The parts of this CTA's share of the rows, in the order of the ranks: eight
  // columns a thread, in at most ITEMS rows.  The CTAs part as soon as all have
  // read, with their stores to come.
  constexpr int ITEMS = (FEW_MOST / 2 * (FN / 8) + FEW_THREADS - 1) / FEW_THREADS;
  static_assert(FEW_THREADS % (FN / 8) == 0, "a thread's rows share its columns");
  const int m0 = p.M * rank / p.ks, m1 = p.M * (rank + 1) / p.ks;
  const int c = threadIdx.x % (FN / 8) * 8, n = unit * FN + c;
  const int cols = min(8, p.N - n);
  float sw[8], bias[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sw[j] = j < cols ? p.sw[n + j] : 0.f;
    bias[j] = p.bias && j < cols ? p.bias[n + j] : 0.f;
  }
  cluster_sync_all();
  float v[ITEMS][8] = {};
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int m = m0 + (int)(threadIdx.x + k * FEW_THREADS) / (FN / 8);
    if (m >= m1 || cols <= 0) continue;
    const uint32_t at = smem_u32(smem) + (uint32_t)(m * FN + c) * 4;
    for (int r = 0; r < p.ks; r += 2) {
      const uint32_t one = cluster_addr(at, r), two = cluster_addr(at, r + 1);
      const float4 a = ld_cluster4(one), b = ld_cluster4(one + 16);
      const float4 d = ld_cluster4(two), e = ld_cluster4(two + 16);
      v[k][0] += a.x; v[k][1] += a.y; v[k][2] += a.z; v[k][3] += a.w;
      v[k][4] += b.x; v[k][5] += b.y; v[k][6] += b.z; v[k][7] += b.w;
      v[k][0] += d.x; v[k][1] += d.y; v[k][2] += d.z; v[k][3] += d.w;
      v[k][4] += e.x; v[k][5] += e.y; v[k][6] += e.z; v[k][7] += e.w;
    }
  }
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int m = m0 + (int)(threadIdx.x + k * FEW_THREADS) / (FN / 8);
    if (m >= m1 || cols <= 0) continue;
    const float sa = s_sa[m];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * sa * sw[j] + bias[j];
    E *y = (E *)p.y + (size_t)m * p.N + n;
    if (p.N % 8 == 0) {
#pragma unroll
      for (int j = 0; j < 8; j += VEC16<E>) {
        float f[VEC16<E>];
#pragma unroll
        for (int i = 0; i < VEC16<E>; ++i) f[i] = v[k][j + i];
        *(uint4 *)(y + j) = pack16(f, (E *)nullptr);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < cols) y[j] = from_f<E>(v[k][j]);
    }
  }
  // no CTA leaves while another may read its part
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// [rows][K] matrix of 8-bit or (f16) 16-bit elements, boxes of `cols` columns
// and `box` rows, 128B-swizzled or not.
bool make_map(CUtensorMap *m, const void *base, int rows, int K, int cols, int box, bool f16,
              bool swizzle) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K * (f16 ? 2 : 1)};
  cuuint32_t bx[2] = {(cuuint32_t)cols, (cuuint32_t)box};
  cuuint32_t es[2] = {1, 1};
  return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
            const_cast<void *>(base), dims, strides, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tile width for `units` pairs that work at once: the least (rounds) x (width +
// 32, a tile's cost apart from its width).
int tile_width(int M, int N, int units) {
  const long mb = (M + ROWS - 1) / ROWS;
  long best = 0;
  int width = 0;
  for (int bn = 256; bn >= 32; bn -= 32) {
    const long tiles = mb * ((N + bn - 1) / bn);
    const long cost = (tiles + units - 1) / units * (bn + 32);
    if (width == 0 || cost < best) {
      best = cost;
      width = bn;
    }
  }
  return width;
}

// CTAs, in clusters of `cluster`, that the GPU runs of a kernel at once.
template <typename Kernel>
cudaError_t ctas_at_once(Kernel kernel, int threads, int smem, int cluster, int *ctas) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms() / cluster * cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
  *ctas = n * cluster;
  return e;
}

cudaError_t launch_widen(const Q8Args &a, cudaStream_t s) {
  const size_t vecs = (size_t)a.M * a.K / 16;
  if ((vecs + 255) / 256 > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  const cudaError_t e =
      launch_k(q8_widen_kernel, dim3((unsigned)((vecs + 255) / 256)), dim3(256), 0, s,
               (const uint4 *)a.aq, vecs, (uint4 *)a.ws);
  prof_mark(KID_Q8_WIDEN, s);
  return e;
}

template <typename E>
cudaError_t mma_t(const Q8Args &a, cudaStream_t s) {
  static int pairs = 0;  // that the GPU runs at once (its SM clusters may have odd ones out)
  static const cudaError_t attr = [] {
    cudaError_t e = cudaFuncSetAttribute(q8_mma_kernel<E>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e == cudaSuccess) e = ctas_at_once(q8_mma_kernel<E>, THREADS, SMEM, 2, &pairs);
    pairs /= 2;
    return e == cudaSuccess && pairs < 1 ? cudaErrorInvalidConfiguration : e;
  }();
  if (attr != cudaSuccess) return attr;
  const cudaError_t e = launch_widen(a, s);
  if (e != cudaSuccess) return e;
  Q8Params p;
  memset(&p, 0, sizeof(p));
  p.M = a.M; p.N = a.N; p.K = a.K; p.sa = a.ascale; p.sw = a.wscale; p.bias = a.bias; p.y = a.y;
  p.status = a.status;
  p.bn = tile_width(a.M, a.N, pairs);
  Q8Maps maps;
  if (!make_map(&maps.a, a.ws, a.M, a.K, BK, BM, true, true) ||
      !make_map(&maps.w, a.wq, a.N, a.K, BK, p.bn / 2, false, false))
    return cudaErrorInvalidValue;
  const long long tiles = (long long)((a.M + ROWS - 1) / ROWS) * ((a.N + p.bn - 1) / p.bn);
  if (tiles > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const int grid = 2 * (tiles < pairs ? (int)tiles : pairs);
  return launch_clusters(q8_mma_kernel<E>, dim3(grid), dim3(THREADS), SMEM, 2, s, maps, p);
}

template <typename E>
cudaError_t few_t(const Q8Args &a, cudaStream_t s) {
  static int at_once[4];  // CTAs in clusters of (1,) 2, 4, 8 that the GPU runs at once
  static const cudaError_t attr = [] {
    cudaError_t e = cudaFuncSetAttribute(q8_few_kernel<E>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, FEW_SMEM);
    for (int i = 1; i < 4 && e == cudaSuccess; ++i)
      e = ctas_at_once(q8_few_kernel<E>, FEW_THREADS, FEW_SMEM, 1 << i, &at_once[i]);
    return e;
  }();
  if (attr != cudaSuccess) return attr;
  cudaError_t e = launch_widen(a, s);
  if (e != cudaSuccess) return e;
  FewParams p;
  memset(&p, 0, sizeof(p));
  p.M = a.M; p.N = a.N; p.K = a.K; p.sa = a.ascale; p.sw = a.wscale; p.bias = a.bias; p.y = a.y;
  p.status = a.status;
  p.box = (a.M + 7) / 8 * 8;
  // the 512 TMEM columns hold two accumulators and four to six stages, the
  // rings in shared memory as many of a and six (no fewer than of the others:
  // the conversion's order of waits) to twelve of w
  p.cols = (a.M + 15) / 16 * 16;
  p.stages = (512 - 2 * p.cols) / (FK / 2);
  if (p.stages > FEW_STAGES) p.stages = FEW_STAGES;
  const int raw = (FEW_RINGS - p.stages * p.box * FK * 2) / (FN * FK);
  p.raw_stages = raw < FEW_RAW ? raw : FEW_RAW;
  // CTAs that share a tile, while all of them run at once: a k-block takes about
  // 600 cycles, the clusters' meetings and the join 5500 (in us, 8 rows and N x K
  // = 2048 x 2048: 9.9 for one CTA a tile, 9.0 for two, 8.4 for four; 8192 x 2048:
  // 10.2 and 10.6; 9728 x 4096: 14.9 and 14.1)
  const int tiles = (a.N + FN - 1) / FN, KT = (a.K + FK - 1) / FK;
  p.ks = 1;
  int best = KT * 600;
  for (int i = 1; i < 4; ++i) {
    const int cost = (KT + (1 << i) - 1) / (1 << i) * 600 + 5500;
    if (((long long)tiles << i) <= at_once[i] && KT >= 1 << i && cost < best) {
      best = cost;
      p.ks = 1 << i;
    }
  }
  Q8Maps maps;
  if (!make_map(&maps.a, a.ws, a.M, a.K, 64, p.box, true, true) ||
      !make_map(&maps.w, a.wq, a.N, a.K, FK, FN, false, true))
    return cudaErrorInvalidValue;
  const int grid = p.ks > 1 ? tiles * p.ks : tiles < num_sms() ? tiles : num_sms();
  return p.ks > 1 ? launch_clusters(q8_few_kernel<E>, dim3(grid), dim3(FEW_THREADS), FEW_SMEM,
                                    p.ks, s, maps, p)
                  : launch_k(q8_few_kernel<E>, dim3(grid), dim3(FEW_THREADS), FEW_SMEM, s, maps, p);
}

template <typename E, int MT>
cudaError_t rows_t(const Q8Args &a, cudaStream_t s) {
  const int groups = (a.N + ROWS_N - 1) / ROWS_N;
  // warps that share K: until 16 warps an SM, while each has 512 bytes a row
  int ks = 1;
  while (ks < 8 && (long long)groups * ks < 16ll * num_sms() && a.K >= ks * 2 * 512) ks *= 2;
  const int per = 8 / ks;
  return launch_k(q8_rows_kernel<E, MT>, dim3((groups + per - 1) / per), dim3(256), 0, s, a.aq,
                  a.wq, a.ascale, a.wscale, a.bias, a.M, a.N, a.K, ks, (E *)a.y);
}

template <typename E, int NT, int MT>
cudaError_t frag_mt(const Q8Args &a, cudaStream_t s) {
  constexpr int WARPS = MT == 2 ? 4 : 8;
  const int tiles = (a.N + MT * 16 - 1) / (MT * 16);
  // warps that share K: until 16 warps an SM, while each has two 64-byte steps
  int ks = 1;
  while (ks < WARPS && (long long)tiles * ks < 16ll * num_sms() && a.K >= ks * 2 * 128) ks *= 2;
  const int per = WARPS / ks;
  return launch_k(q8_frag_kernel<E, NT, MT, WARPS>, dim3((tiles + per - 1) / per),
                  dim3(WARPS * 32), 0, s, (const uint4 *)a.aq, a.wq, a.ascale, a.wscale, a.bias,
                  a.M, a.N, a.K, ks, (E *)a.y);
}

template <typename E, int NT>
cudaError_t frag_t(const Q8Args &a, cudaStream_t s) {
  // 32 weight rows a warp where that leaves eight warps an SM: rows of a are
  // widened half as often, in half as many warps (us, 16 and 32 weight rows, at
  // 8192 x 2048 | 9728 x 2048 | 14336 x 2048 | 16000 x 1024 | 50001 x 512: 8 rows 6.3 |
  // 7.1 | 8.8 | 6.6 | 9.6 and 7.6 | 8.0 | 9.0 | 6.4 | 8.8; 16 rows 8.6 | 8.5 | 11.1 |
  // 9.1 | 12.6 and 9.0 | 9.3 | 10.6 | 7.6 | 13.9: the two cross about there)
  return a.N >= 64 * num_sms() ? frag_mt<E, NT, 2>(a, s) : frag_mt<E, NT, 1>(a, s);
}

// Whether a batch of decoded rows is multiplied in fragments: it starts and ends
// sooner, but rows of a are widened again in every warp.  Measured, us at N x K =
// 2048 x 2048 | 8192 x 2048 | 4096 x 4096 | 8192 x 4096 | 14336 x 4096 | 50001 x
// 2048 | 14336 x 16384 (weights from HBM; the floors, N x K bytes, are 0.6 | 2.5 |
// 2.5 | 4.9 | 8.6 | 15 | 35):
//   M 1    rows 2.4 | 4.5 | 4.6 | 7.3 | 11.8 | 19.0 | 41
//          few  7.8 | 9.7 | 10.0 | 12.8 | 15.1 | 24.1 | 43
//   M 4    rows 3.1 | 6.8 | 6.9 | 9.1 | 13.1 | 22.2 | 42
//          few  7.9 | 9.7 | 10.1 | 12.8 | 15.1 | 23.5 | 43
//   M 8    frag 3.6 | 6.4 | 7.0 | 10.4 | 16.8 | 24.3 | 64
//          few  7.9 | 9.8 | 10.3 | 12.6 | 15.5 | 23.7 | 43
//   M 16   frag 4.3 | 8.6 | 8.1 | 12.8 | 18.0 | 33.0 | 61
//          few  8.1 | 9.9 | 10.5 | 12.9 | 15.5 | 24.2 | 44
//   M 32   frag 5.3 | 12.5 | 11.3 | 20.6 | 36.5 | 68 | 151
//          few  8.6 | 10.1 | 11.0 | 13.5 | 15.4 | 24.2 | 45
//   M 64   few  9.8 | 10.8 | 12.5 | 13.9 | 16.5 | 25.5 | 49
//          pair 12.3 | 14.3 | 19.8 | 21.2 | 26.7 | 39.4 | 80
//   M 128  few  12.6 | 12.7 | 15.5 | 16.9 | 19.1 | 31.5 | 58
//          pair 12.2 | 14.8 | 20.1 | 21.8 | 28.0 | 43.0 | 82
// (Up to four rows stay with the simplest kernel.  Columns count too: 17 to 32
// rows of 50001 x 256 take the fragments 16 to 18 us, few 10.5.  And 33 to 64
// rows at 1000 x 1024 | 2048 x 2048 | 4096 x 2048 | 2048 x 4096 | 8192 x 1024: 48
// rows in fragments 3.9 | 6.5 | 8.6 | 10.1 | 10.7, few 6.9 | 9.2 | 10.5 | 10.8 |
// 8.4; 64 rows 4.9 | 7.8 | 10.5 | 12.0 | 13.0 and 7.0 | 9.8 | 11.1 | 11.4 | 8.7.)
// And k: at most eight warps of one CTA share it in the fragments, clusters of
// eight CTAs in few.  N x K = 1000 x 3584 | 2048 x 8192 | 1000 x 8192 | 1000 x 16384 |
// 128 x 65536, fragments and few: 8 rows 5.7 | 10.4 | 10.1 | 18.7 | 66 and 8.0 |
// 11.3 | 9.6 | 11.6 | 22; 16 rows 6.1 | 11.2 | 10.9 | 19.5 | 71 and 7.9 | 11.5 | 9.8 |
// 11.8 | 23; 32 rows 7.5 | 13.8 | 13.6 | 24.5 | 89 and 8.7 | 12.0 | 10.5 | 12.7 | 24;
// 48 rows 9.1 | 16.6 | 16.3 | 29 | 107 and 9.5 | 12.9 | 11.5 | 13.8 | 26; 64 rows
// 11.4 | 20.3 | 20.1 | 37 | 131 and 10.3 | 13.8 | 12.5 | 14.8 | 27.
bool in_fragments(int M, int N, int K) {
  const long long bytes = (long long)N * K;
  return M <= 8    ? K <= 8192 && bytes < 3ll << 24
         : M <= 16 ? K <= 8192 && bytes < 1ll << 25
         : M <= 32 ? K <= 4096 && N <= 8192 && bytes < 1ll << 24
                   : M <= 64 && K <= (M <= 48 ? 4096 : 2048) && N <= 4096 && bytes <= 1ll << 23;
}

template <typename E>
cudaError_t matmul_t(const Q8Args &a, cudaStream_t s) {
  if (a.M == 1) return rows_t<E, 1>(a, s);
  if (a.M == 2) return rows_t<E, 2>(a, s);
  if (a.M <= ROWS_MAX) return rows_t<E, 4>(a, s);
  if (in_fragments(a.M, a.N, a.K))
    return a.M <= 8    ? frag_t<E, 1>(a, s)
           : a.M <= 16 ? frag_t<E, 2>(a, s)
           : a.M <= 32 ? frag_mt<E, 4, 1>(a, s)
           : a.M <= 48 ? frag_mt<E, 6, 1>(a, s)
                       : frag_mt<E, 8, 1>(a, s);
  return a.M <= FEW_MOST ? few_t<E>(a, s) : mma_t<E>(a, s);
}

}  // namespace

size_t q8_scratch(int M, int N, int K) {
  // a in fp16
  return M <= ROWS_MAX || in_fragments(M, N, K) ? 0 : ((size_t)M * K * 2 + 255) / 256 * 256;
}

cudaError_t launch_q8_matmul(const Q8Args &a, cudaStream_t s) {
  const cudaError_t e = a.dtype == TWELL_BF16 ? matmul_t<bf16>(a, s) : matmul_t<float>(a, s);
  prof_mark(KID_Q8_MATMUL, s);
  return e;
}

}  // namespace twell

#ifdef TWELL_TEST_HOOKS
extern "C" int twell_test_q8_pairs(unsigned *ended, unsigned *early) {
  unsigned n[2] = {0, 0};
  const unsigned zero[2] = {0, 0};
  if (cudaMemcpyFromSymbol(n, twell::test_pairs, sizeof(n)) != cudaSuccess ||
      cudaMemcpyToSymbol(twell::test_pairs, zero, sizeof(zero)) != cudaSuccess)
    return TWELL_ERR_CUDA;
  *ended = n[0];
  *early = n[1];
  return TWELL_OK;
}
#endif
