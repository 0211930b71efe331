// q8.cu -- product of 8-bit rows: y[m][n] = sa[m] sw[n] sum_k a[m][k] w[n][k]
// (+ bias[n]).
//
// sm_103a has no fast 8-bit integer tensor path, but an 8-bit integer is
// exact in fp16, its products are exact in fp32, and so is their sum while
// it stays below 2^24: the fp16 tensor cores (tcgen05 kind::f16, fp32
// accumulators in TMEM) do this product at twice the width and full speed.
// The operands stay 8-bit in memory and are widened on their way through
// shared memory.
//
// By the rows of a (matmul_t has the rule and the measurements):
//   a decoded row or four   q8_rows_kernel: dp4a, exact int32 sums
//   a batch of them         q8_frag_kernel: the weights are widened in
//                           registers and used up there (m16n8k16)
//   up to 128 rows          q8_mma_kernel: TMA brings 8-bit tiles, warps
//                           widen them into the MMA's shared-memory layout,
//                           one lane issues tcgen05.mma, four warps read TMEM
//   more                    q8_pair_kernel: the same over CTA pairs
#include <cuda_fp16.h>
#include <string.h>

#include "common.cuh"
#include "lm_kernels.h"
#include "tcgen05.cuh"
#include "vec16.cuh"

namespace twell {

namespace {

// ---- few rows ----------------------------------------------------------------
constexpr int ROWS_MAX = 4;  // rows of a that q8_rows_kernel takes
constexpr int ROWS_N = 4;    // weight rows a warp reads together

// A group of KS warps takes ROWS_N weight rows and splits K; MT rows of a
// (M <= MT) are read again by every warp, from L1.  Sums are integers, so
// the split leaves no trace.
template <typename E, int MT>
__global__ void __launch_bounds__(256)
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
#pragma unroll 2
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
// L1, was slower: 47 against 33 us at 16 x 50001 x 2048).  A tile's KS warps
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
__global__ void __launch_bounds__(WARPS * 32)
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
constexpr int GROUPS = 4, GROUP = 4;            // conversion groups, warps of a group
constexpr int THREADS = 32 * (6 + GROUPS * GROUP);  // TMA, MMA, 4 epilogue, conversion
constexpr int F16_STAGES_MAX = 8, RAW_STAGES_MAX = 24;
constexpr int ACC_COLS = 256;                   // TMEM columns of one accumulator
constexpr int EPI_PITCH = 33;                   // 32-bit words of an epilogue staging row

struct Q8Maps {
  CUtensorMap a, w;
};

// Shape of the pipeline (the same for every CTA).
struct Q8Plan {
  int bn;         // output columns per tile (a multiple of 16, at most 256)
  int ar;         // rows of a that a tile holds (a multiple of 16, at most 128)
  int raw, f16;   // stages (a k-block each)
  int raw_bytes, f16_bytes;
};

struct Q8Params {
  int M, N, K;
  const float *sa, *sw, *bias;
  void *y;
  int32_t *status;
  Q8Plan pl;
};

__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// One warp's 32 accumulator rows (TMEM lane = row, from row m0 on) of a tile
// of bn columns from n0 on: scaled, rounded, and stored through shared memory
// so that one instruction writes 128 consecutive bytes of a row whatever its
// alignment.
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

__device__ __forceinline__ void store_tile(const Q8Params &p, float *y, uint32_t acc, int m0,
                                           int n0, float sa, const float *s_sw, float *stage) {
  const int lane = threadIdx.x & 31, cols = min(p.pl.bn, p.N - n0), rows = min(32, p.M - m0);
  for (int c0 = 0; c0 < cols; c0 += 32) {
    float v[32];
    tmem_ld32(acc + c0, v);
    scale32(v, sa, s_sw + c0, s_sw + 256 + c0);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i) stage[lane * EPI_PITCH + i] = v[i];
    __syncwarp();
    float *dst = y + (size_t)m0 * p.N + n0 + c0 + lane;
    if (c0 + lane < cols)
#pragma unroll 4
      for (int r = 0; r < rows; ++r) dst[(size_t)r * p.N] = stage[r * EPI_PITCH + lane];
  }
}

// bf16: pairs of elements as they lie in aligned 4-byte words of y.  With an
// odd N every other row starts in the upper half of a word; such a row's
// pairs are (-1, 0), (1, 2), ...: its thread packs them so, carrying one
// element from block to block, and only a tile's first and last words are
// stored by halves.
__device__ __forceinline__ void store_tile(const Q8Params &p, bf16 *y, uint32_t acc, int m0,
                                           int n0, float sa, const float *s_sw, float *stage_f) {
  uint32_t *stage = (uint32_t *)stage_f;
  const int lane = threadIdx.x & 31, cols = min(p.pl.bn, p.N - n0), rows = min(32, p.M - m0);
  const int odd_n = p.N & 1;                  // (n0 is even)
  const bool odd = (odd_n & (m0 + lane)) != 0;
  float carry = 0.f;
  if (p.N % 8 == 0) {
    // 16-byte aligned rows: each thread stores its own (a last tile's epilogue
    // is over sooner: 18.7 against 21.6 us at 300 x 8192 x 2048)
    for (int c0 = 0; c0 < cols; c0 += 32) {
      float v[32];
      tmem_ld32(acc + c0, v);
      scale32(v, sa, s_sw + c0, s_sw + 256 + c0);
      uint4 *dst = (uint4 *)(y + (size_t)(m0 + lane) * p.N + n0 + c0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane < rows && c0 + 8 * i < cols)
          dst[i] = make_uint4(pack_bf2(v[8 * i], v[8 * i + 1]), pack_bf2(v[8 * i + 2], v[8 * i + 3]),
                              pack_bf2(v[8 * i + 4], v[8 * i + 5]),
                              pack_bf2(v[8 * i + 6], v[8 * i + 7]));
    }
    return;
  }
  for (int c0 = 0; c0 < cols; c0 += 64) {
    float v[64];
    tmem_ld32(acc + c0, *(float(*)[32])v);
    if (c0 + 32 < p.pl.bn) tmem_ld32(acc + c0 + 32, *(float(*)[32])(v + 32));
    scale32(v, sa, s_sw + c0, s_sw + 256 + c0);
    scale32(v + 32, sa, s_sw + c0 + 32, s_sw + 256 + c0 + 32);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; ++j)
      stage[lane * EPI_PITCH + j] = pack_bf2(odd ? (j ? v[2 * j - 1] : carry) : v[2 * j],
                                             odd ? v[2 * j] : v[2 * j + 1]);
    carry = v[63];
    __syncwarp();
    bf16 *dst = y + (size_t)m0 * p.N + n0 + c0 + 2 * lane;
    if (c0 > 0 && c0 + 64 < cols) {
#pragma unroll 4
      for (int r = 0; r < rows; ++r)
        *(uint32_t *)(dst + (size_t)r * p.N - (odd_n & (m0 + r))) = stage[r * EPI_PITCH + lane];
    } else {
      for (int r = 0; r < rows; ++r) {
        const int o = odd_n & (m0 + r), c = c0 + 2 * lane - o;  // column of the word's lower half
        const uint32_t w = stage[r * EPI_PITCH + lane];
        bf16 *d = dst + (size_t)r * p.N - o;
        if (c >= 0 && c + 1 < cols) {
          *(uint32_t *)d = w;
        } else if (c >= 0 && c < cols) {
          *(uint16_t *)d = (uint16_t)w;
        } else if (c == -1) {
          *(uint16_t *)(d + 1) = (uint16_t)(w >> 16);
        }
      }
    }
  }
  // the last element of a shifted row whose columns fill the last block
  if (odd && lane < rows && cols % 64 == 0)
    y[(size_t)(m0 + lane) * p.N + n0 + cols - 1] = __float2bfloat16_rn(carry);
}

// Scale and bias of a tile's columns, staged by the 128 epilogue threads.
__device__ __forceinline__ void stage_columns(const Q8Params &p, int n0, float *s_sw, int et) {
  epi_bar();
  for (int c = et; c < p.pl.bn; c += 128) {
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

// After an abort no copy may be in flight when the CTA exits: waits (bounded)
// for the last load that was issued into each stage of a ring.
__device__ __forceinline__ void drain_ring(uint32_t full, int S, long issued) {
  for (int s = 0; s < S && s < issued; ++s) {
    const uint32_t par = (uint32_t)(((issued - 1 - s) / S) & 1);
    const uint64_t t0 = global_timer();
    while (!mbar_try(full + 8 * s, par) && global_timer() - t0 < DRAIN_LIMIT_NS) {
    }
  }
}

// Address part of the swizzled operand descriptors (sw128_desc): adding to
// the low word moves the start, 16 bytes a unit.
__device__ __forceinline__ uint64_t desc_at(uint32_t saddr) { return sw128_desc(saddr, 16, 1024); }

template <typename E>
__global__ void __launch_bounds__(THREADS, 1)
q8_mma_kernel(const __grid_constant__ Q8Maps maps, const __grid_constant__ Q8Params p) {
  pdl_begin();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const Q8Plan pl = p.pl;
  // An fp16 stage holds the ar rows of a, then the bn rows of w; the MMA's
  // 128 rows of a run into those of w when ar < 128 (accumulator rows that
  // are not stored).
  uint8_t *f16 = smem;                                   // [f16][A ar rows, W bn rows] x 128 B
  uint8_t *raw = smem + pl.f16 * pl.f16_bytes;           // [raw][A ar rows, W bn rows] x 64 B
  float *s_epi = (float *)(raw + pl.raw * pl.raw_bytes); // [4][32][EPI_PITCH]
  float *s_sw = s_epi + 4 * 32 * EPI_PITCH;              // [2][256] scale, bias of the columns
  __shared__ uint64_t bars[2 * RAW_STAGES_MAX + 2 * F16_STAGES_MAX + 5];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;
  const uint32_t rfull = smem_u32(bars), rempty = rfull + 8 * RAW_STAGES_MAX;
  const uint32_t ffull = rempty + 8 * RAW_STAGES_MAX, fempty = ffull + 8 * F16_STAGES_MAX;
  const uint32_t tfull = fempty + 8 * F16_STAGES_MAX, tempty = tfull + 16, mma_done = tempty + 16;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  const int mb = (p.M + BM - 1) / BM, nb = (p.N + pl.bn - 1) / pl.bn;
  const int tiles = mb * nb;  // M-blocks innermost: the CTAs in flight share few weight tiles
  const int KT = (p.K + BK - 1) / BK;

  if (threadIdx.x == 0) {
    for (int i = 0; i < pl.raw; ++i) {
      mbar_init(rfull + 8 * i, 1);
      mbar_init(rempty + 8 * i, GROUP);
    }
    for (int i = 0; i < pl.f16; ++i) {
      mbar_init(ffull + 8 * i, GROUP);
      mbar_init(fempty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, 4);
    }
    mbar_init(mma_done, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem)),
                 "r"(2 * ACC_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    const bool issues = elect_one();
    const uint32_t raw0 = smem_u32(raw);
    int st = 0;
    uint32_t ph = 0;
    long issued = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const int m0 = (t % mb) * BM, n0 = (t / mb) * pl.bn;
      for (int kt = 0; kt < KT; ++kt) {
        ok = warp_wait(rempty + 8 * st, ph ^ 1, abort_flag, p.status);
        if (!ok) break;
        const uint32_t bar = rfull + 8 * st, dst = raw0 + st * pl.raw_bytes;
        if (issues) {
          mbar_expect_tx(bar, (uint32_t)pl.raw_bytes);
          tma_load_2d(dst, &maps.a, kt * BK, m0, bar);
          tma_load_2d(dst + pl.ar * BK, &maps.w, kt * BK, n0, bar);
        }
        __syncwarp();
        ++issued;
        if (++st == pl.raw) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok) drain_ring(rfull, pl.raw, issued);
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer --
    {
      const bool issues = elect_one();
      const uint32_t idesc = make_idesc(BM, pl.bn, false, false, true);
      const uint64_t ad0 = desc_at(smem_u32(f16));
      const uint32_t w_off = (uint32_t)(pl.ar * 128) >> 4;
      int st = 0, lt = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++lt) {
        const int buf = lt & 1;
        ok = warp_wait(tempty + 8 * buf, ((uint32_t)(lt >> 1) & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * ACC_COLS);
        for (int kt = 0; kt < KT; ++kt) {
          ok = warp_wait(ffull + 8 * st, ph, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = ad0 + (uint32_t)(st * pl.f16_bytes >> 4), wd = ad + w_off;
          if (issues) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)  // 32 bytes of a row a step
              mma_bf16(acc, ad + 2 * kk, wd + 2 * kk, idesc, (kt > 0 || kk > 0) ? 1u : 0u);
            mma_commit(fempty + 8 * st);
          }
          __syncwarp();
          if (++st == pl.f16) {
            st = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        if (issues) mma_commit(tfull + 8 * buf);
        __syncwarp();
      }
      // all MMAs issued by this thread are complete before TMEM is freed
      if (issues) mma_commit(mma_done);
      const uint64_t t0 = global_timer();
      while (!mbar_try(mma_done, 0) && global_timer() - t0 < DRAIN_LIMIT_NS) {
      }
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue --
    const int q = warp & 3;  // TMEM lane quadrant of this warp
    const int et = threadIdx.x - 64;
    float *stage = s_epi + q * 32 * EPI_PITCH;
    int lt = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++lt) {
      const int m0 = (t % mb) * BM, n0 = (t / mb) * pl.bn;
      const int buf = lt & 1;
      const int m = m0 + q * 32 + lane;
      stage_columns(p, n0, s_sw, et);
      const float sa = m < p.M ? p.sa[m] : 0.f;
      const bool ok = epi_all(mbar_wait(tfull + 8 * buf, (uint32_t)(lt >> 1) & 1, abort_flag,
                                        p.status));
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * ACC_COLS);
      if (m0 + q * 32 < p.M)  // (uniform for the warp)
        store_tile(p, (E *)p.y, acc, m0 + q * 32, n0, sa, s_sw, stage);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty + 8 * buf);
    }
  } else {
    // ---------------------------------------------------------- conversion --
    // Four groups of warps take the k-blocks in turn.
    const int group = (warp - 6) / GROUP, ct = (threadIdx.x - 192) % (32 * GROUP);
    const int vecs = (pl.ar + pl.bn) * (BK / 16);  // 16-byte vectors of a k-block
    const int mine = (tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    Ring f(group, pl.f16), r(group, pl.raw);
    for (long it = group; it < (long)mine * KT; it += GROUPS) {
      if (!warp_wait(rfull + 8 * r.at, r.phase, abort_flag, p.status)) break;
      if (!warp_wait(fempty + 8 * f.at, f.phase ^ 1, abort_flag, p.status)) break;
      widen_rows<32 * GROUP>(raw + r.at * pl.raw_bytes, f16 + f.at * pl.f16_bytes, ct, vecs);
      fence_async_proxy();  // the MMA reads through the async proxy
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ffull + 8 * f.at);
        mbar_arrive(rempty + 8 * r.at);
      }
      f.next<GROUPS>(pl.f16);
      r.next<GROUPS>(pl.raw);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(2 * ACC_COLS)
                 : "memory");
  }
}

// ---- tensor cores, CTA pairs ----------------------------------------------------
// More than 128 rows of a: two CTAs (one cluster) share a 256 x bn tile.
// Each holds 128 rows of a and bn / 2 rows of w, the leader issues
// cta_group::2 MMAs over both, and each CTA stores its 128 rows.  a is
// widened once by q8_widen_kernel and comes by TMA as fp16; w is widened
// here, each row once per CTA pair: per k-block an SM then moves 64 KB through
// shared memory (w in 8 bits twice and in fp16 once, a once, the MMA's reads)
// where one CTA that widened both operands for its own 128 x 256 tile would
// move 144 KB for the same multiplications, and shared memory, not the
// tensor cores, was its bound.
//
// A conversion warp's stores, their fence and its arrival take about 2000
// cycles from end to end, four times a k-block's MMAs, so four groups of
// warps take the k-blocks in turn.  They arrive at a barrier of their own
// CTA and one thread passes that on to the leader: a release across the
// cluster by the storing warps themselves waits for their stores once more
// (704 TFLOP/s at M 8192, N 14336, K 4096 with two groups that did).
constexpr int P_AS = 5, P_BS = 4, P_RS = 6;     // stages: a, w in fp16, w in 8 bits
constexpr int P_GROUPS = 4, P_GROUP = 2;        // conversion groups, warps of a group
constexpr int P_THREADS = 32 * (8 + P_GROUPS * P_GROUP);
constexpr int P_TILE = 128 * 128;               // bytes of an fp16 stage (a or w)
constexpr int P_RAW = 128 * BK;
constexpr int P_SMEM = 1024 + P_AS * P_TILE + P_BS * P_TILE + P_RS * P_RAW +
                       4 * 32 * EPI_PITCH * 4 + 2 * 256 * 4;

// fp16 copy of a.
__global__ void __launch_bounds__(256)
q8_widen_kernel(const uint4 *a, size_t vecs, uint4 *out) {
  pdl_begin();
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= vecs) return;
  uint4 lo, hi;
  widen16(ldg_stream<L2_FIRST>(a + i), lo, hi);
  out[2 * i] = lo;
  out[2 * i + 1] = hi;
}

template <typename E>
__global__ void __launch_bounds__(P_THREADS, 1)
q8_pair_kernel(const __grid_constant__ Q8Maps maps, const __grid_constant__ Q8Params p) {
  pdl_begin();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sa16 = smem, *sw16 = sa16 + P_AS * P_TILE, *raw = sw16 + P_BS * P_TILE;
  float *s_epi = (float *)(raw + P_RS * P_RAW);
  float *s_sw = s_epi + 4 * 32 * EPI_PITCH;
  // Barriers of this CTA: a stage is full, a stage is free again.  Barriers
  // of the leader, at which both CTAs arrive: a k-block's operands are ready,
  // an accumulator has been read (tempty).
  __shared__ uint64_t bars[2 * P_AS + 3 * P_BS + 2 * P_RS + 5];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;
  const uint32_t afull = smem_u32(bars), aempty = afull + 8 * P_AS;
  const uint32_t wfull = aempty + 8 * P_AS, wempty = wfull + 8 * P_BS, ready = wempty + 8 * P_BS;
  const uint32_t rfull = ready + 8 * P_BS, rempty = rfull + 8 * P_RS;
  const uint32_t tfull = rempty + 8 * P_RS, tempty = tfull + 16, mma_done = tempty + 16;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x & 1);  // in the pair (clusters are consecutive CTAs)
  const int bn = p.pl.bn, half = bn / 2;

  const int mb = (p.M + 2 * BM - 1) / (2 * BM), nb = (p.N + bn - 1) / bn;
  const int tiles = mb * nb;  // M-blocks innermost: the pairs in flight share few weight tiles
  const int KT = (p.K + BK - 1) / BK;
  const int pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;
  const long its = (long)((tiles - pair + pairs - 1) / pairs) * KT;  // k-blocks of this pair

  if (threadIdx.x == 0) {
    for (int i = 0; i < P_AS; ++i) {
      mbar_init(afull + 8 * i, 1);
      mbar_init(aempty + 8 * i, 1);
    }
    for (int i = 0; i < P_BS; ++i) {
      mbar_init(wfull + 8 * i, P_GROUP);
      mbar_init(wempty + 8 * i, 1);
      mbar_init(ready + 8 * i, 2);
    }
    for (int i = 0; i < P_RS; ++i) {
      mbar_init(rfull + 8 * i, 1);
      mbar_init(rempty + 8 * i, P_GROUP);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, 8);
    }
    mbar_init(mma_done, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem)),
                 "r"(2 * ACC_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == 0 || warp == 6) {
    // ------------------------------- TMA producers: w in 8 bits; a in fp16 --
    const bool issues = elect_one();
    const bool is_w = warp == 0;
    const uint32_t full = is_w ? rfull : afull, empty = is_w ? rempty : aempty;
    const uint32_t dst0 = smem_u32(is_w ? raw : sa16), step = is_w ? P_RAW : P_TILE;
    const int S = is_w ? P_RS : P_AS, bytes = is_w ? half * BK : P_TILE;
    const CUtensorMap *map = is_w ? &maps.w : &maps.a;
    int st = 0;
    uint32_t ph = 0;
    long issued = 0;
    bool ok = true;
    for (int t = pair; t < tiles && ok; t += pairs) {
      const int row = is_w ? (t / mb) * bn + rank * half : (t % mb) * 2 * BM + rank * BM;
      for (int kt = 0; kt < KT; ++kt) {
        ok = warp_wait(empty + 8 * st, ph ^ 1, abort_flag, p.status);
        if (!ok) break;
        if (issues) {
          mbar_expect_tx(full + 8 * st, (uint32_t)bytes);
          tma_load_2d(dst0 + st * step, map, kt * BK, row, full + 8 * st);
        }
        __syncwarp();
        ++issued;
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok) drain_ring(full, S, issued);
  } else if (warp == 7) {
    // ------------- tells the leader that this CTA's operands have arrived --
    if (lane == 0) {
      const uint32_t to = cluster_addr(ready, 0);
      Ring a(0, P_AS), w(0, P_BS);
      for (long it = 0; it < its; ++it) {
        if (!mbar_wait(afull + 8 * a.at, a.phase, abort_flag, p.status) ||
            !mbar_wait(wfull + 8 * w.at, w.phase, abort_flag, p.status))
          break;
        mbar_arrive_cluster(to + 8 * w.at);
        a.next(P_AS);
        w.next(P_BS);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer --
    if (rank == 0) {
      const bool issues = elect_one();
      const uint32_t idesc = make_idesc(2 * BM, bn, false, false, true);
      const uint64_t ad0 = desc_at(smem_u32(sa16)), wd0 = desc_at(smem_u32(sw16));
      Ring a(0, P_AS), w(0, P_BS);
      int lt = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, ++lt) {
        const int buf = lt & 1;
        ok = warp_wait(tempty + 8 * buf, ((uint32_t)(lt >> 1) & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * ACC_COLS);
        for (int kt = 0; kt < KT; ++kt) {
          ok = warp_wait(ready + 8 * w.at, w.phase, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = ad0 + (uint32_t)(a.at * (P_TILE >> 4));
          const uint64_t wd = wd0 + (uint32_t)(w.at * (P_TILE >> 4));
          if (issues) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_f16_pair(acc, ad + 2 * kk, wd + 2 * kk, idesc, (kt > 0 || kk > 0) ? 1u : 0u);
            mma_commit_pair(aempty + 8 * a.at);
            mma_commit_pair(wempty + 8 * w.at);
          }
          __syncwarp();
          a.next(P_AS);
          w.next(P_BS);
        }
        if (!ok) break;
        if (issues) mma_commit_pair(tfull + 8 * buf);
        __syncwarp();
      }
      // all MMAs issued by this thread are complete before TMEM is freed
      if (issues) mma_commit_pair(mma_done);
      const uint64_t t0 = global_timer();
      while (!mbar_try(mma_done, 0) && global_timer() - t0 < DRAIN_LIMIT_NS) {
      }
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue --
    const int q = warp & 3;  // TMEM lane quadrant of this warp
    float *stage = s_epi + q * 32 * EPI_PITCH;
    const uint32_t free = cluster_addr(tempty, 0);
    int lt = 0;
    for (int t = pair; t < tiles; t += pairs, ++lt) {
      const int m0 = (t % mb) * 2 * BM + rank * BM + q * 32, n0 = (t / mb) * bn;
      const int buf = lt & 1;
      stage_columns(p, n0, s_sw, threadIdx.x - 64);
      const float sa = m0 + lane < p.M ? p.sa[m0 + lane] : 0.f;
      const bool ok = epi_all(mbar_wait(tfull + 8 * buf, (uint32_t)(lt >> 1) & 1,
                                                abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
      if (m0 < p.M)  // (uniform for the warp)
        store_tile(p, (E *)p.y, tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * ACC_COLS), m0,
                   n0, sa, s_sw, stage);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(free + 8 * buf);
    }
  } else {
    // ---------------------------------------------------------- conversion --
    const int group = (warp - 8) / P_GROUP, ct = (threadIdx.x - 256) % (32 * P_GROUP);
    const int vecs = half * (BK / 16);
    Ring w(group, P_BS), r(group, P_RS);
    for (long it = group; it < its; it += P_GROUPS) {
      if (!warp_wait(rfull + 8 * r.at, r.phase, abort_flag, p.status)) break;
      if (!warp_wait(wempty + 8 * w.at, w.phase ^ 1, abort_flag, p.status)) break;
      widen_rows<32 * P_GROUP>(raw + r.at * P_RAW, sw16 + w.at * P_TILE, ct, vecs);
      fence_async_proxy();  // the MMA reads through the async proxy
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(wfull + 8 * w.at);
        mbar_arrive(rempty + 8 * r.at);
      }
      w.next<P_GROUPS>(P_BS);
      r.next<P_GROUPS>(P_RS);
    }
  }

  // neither CTA leaves while the other may reach its shared memory or TMEM
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(2 * ACC_COLS)
                 : "memory");
  }
}

// [rows][K] matrix of 8-bit or (f16) 16-bit elements, boxes of 64 columns and
// `box` rows; 16-bit boxes 128B-swizzled, as the MMA reads them.
bool make_map(CUtensorMap *m, const void *base, int rows, int K, int box, bool f16) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K * (f16 ? 2 : 1)};
  cuuint32_t bx[2] = {BK, (cuuint32_t)box};
  cuuint32_t es[2] = {1, 1};
  return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
            const_cast<void *>(base), dims, strides, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            f16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int SMEM_FIXED = 1024 + 4 * 32 * EPI_PITCH * 4 + 2 * 256 * 4;
constexpr int SMEM_MAX = 225 * 1024;

// Tile width for `units` CTAs or pairs that work at once: the least (rounds)
// x (width + `fixed`, a tile's cost apart from its width).
int tile_width(int M, int N, int rows, int units, int step, int fixed) {
  const long mb = (M + rows - 1) / rows;
  long best = 0;
  int width = 0;
  for (int bn = 256; bn >= step; bn -= step) {
    const long tiles = mb * ((N + bn - 1) / bn);
    const long cost = (tiles + units - 1) / units * (bn + fixed);
    if (width == 0 || cost < best) {
      best = cost;
      width = bn;
    }
  }
  return width;
}

Q8Plan plan_of(int M, int N) {
  Q8Plan pl;
  pl.ar = M > BM ? BM : (M + 15) / 16 * 16;
  pl.bn = tile_width(M, N, BM, num_sms(), 16, 32);
  pl.raw_bytes = (pl.ar + pl.bn) * BK;
  pl.f16_bytes = (pl.ar + pl.bn) * 128;
  // fp16 stages while the 8-bit stages keep a third of shared memory (the
  // MMA's reach past the last fp16 stage stays inside it: a 128-row tile is
  // 16 KB)
  const int room = SMEM_MAX - SMEM_FIXED;
  pl.f16 = F16_STAGES_MAX;
  while (pl.f16 > 2 && room - pl.f16 * pl.f16_bytes < room / 3) --pl.f16;
  pl.raw = (room - pl.f16 * pl.f16_bytes) / pl.raw_bytes;
  if (pl.raw > RAW_STAGES_MAX) pl.raw = RAW_STAGES_MAX;
  return pl;
}

template <typename E>
cudaError_t mma_t(const Q8Args &a, cudaStream_t s) {
  Q8Params p;
  p.M = a.M; p.N = a.N; p.K = a.K; p.sa = a.ascale; p.sw = a.wscale; p.bias = a.bias; p.y = a.y;
  p.status = a.status;
  p.pl = plan_of(a.M, a.N);
  Q8Maps maps;
  if (!make_map(&maps.a, a.aq, a.M, a.K, p.pl.ar, false) ||
      !make_map(&maps.w, a.wq, a.N, a.K, p.pl.bn, false))
    return cudaErrorInvalidValue;
  static const cudaError_t attr = cudaFuncSetAttribute(
      q8_mma_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
  if (attr != cudaSuccess) return attr;
  const long long tiles =
      (long long)((a.M + BM - 1) / BM) * ((a.N + p.pl.bn - 1) / p.pl.bn);
  if (tiles > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const int grid = tiles < num_sms() ? (int)tiles : num_sms();
  const size_t smem =
      SMEM_FIXED + (size_t)p.pl.f16 * p.pl.f16_bytes + (size_t)p.pl.raw * p.pl.raw_bytes;
  return launch_k(q8_mma_kernel<E>, dim3(grid), dim3(THREADS), smem, s, maps, p);
}

// Rows of a from which CTA pairs are used.
constexpr int PAIR_MIN = 129;

template <typename E>
cudaError_t pair_t(const Q8Args &a, cudaStream_t s) {
  static int most = 0;  // pairs that the GPU runs at once (its SM clusters may have odd ones out)
  static const cudaError_t attr = [] {
    cudaError_t e = cudaFuncSetAttribute(q8_pair_kernel<E>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, P_SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (num_sms() / 2));
    cfg.blockDim = dim3(P_THREADS);
    cfg.dynamicSmemBytes = P_SMEM;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&most, q8_pair_kernel<E>, &cfg);
    return e == cudaSuccess && most < 1 ? cudaErrorInvalidConfiguration : e;
  }();
  if (attr != cudaSuccess) return attr;
  const size_t vecs = (size_t)a.M * a.K / 16;
  if ((vecs + 255) / 256 > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  const cudaError_t e =
      launch_k(q8_widen_kernel, dim3((unsigned)((vecs + 255) / 256)), dim3(256), 0, s,
               (const uint4 *)a.aq, vecs, (uint4 *)a.ws);
  if (e != cudaSuccess) return e;
  prof_mark(KID_Q8_WIDEN, s);
  Q8Params p;
  memset(&p, 0, sizeof(p));
  p.M = a.M; p.N = a.N; p.K = a.K; p.sa = a.ascale; p.sw = a.wscale; p.bias = a.bias; p.y = a.y;
  p.status = a.status;
  p.pl.bn = tile_width(a.M, a.N, 2 * BM, most, 32, 32);
  Q8Maps maps;
  if (!make_map(&maps.a, a.ws, a.M, a.K, BM, true) ||
      !make_map(&maps.w, a.wq, a.N, a.K, p.pl.bn / 2, false))
    return cudaErrorInvalidValue;
  const long long tiles =
      (long long)((a.M + 2 * BM - 1) / (2 * BM)) * ((a.N + p.pl.bn - 1) / p.pl.bn);
  if (tiles > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const int grid = 2 * (tiles < most ? (int)tiles : most);
  return launch_clusters(q8_pair_kernel<E>, dim3(grid), dim3(P_THREADS), P_SMEM, 2, s, maps, p);
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
  // 32 weight rows a warp where that leaves eight warps an SM (rows of a are
  // widened half as often: 22.6 against 28.4 us at 1 x 50001 x 2048)
  return a.N >= 64 * num_sms() ? frag_mt<E, NT, 2>(a, s) : frag_mt<E, NT, 1>(a, s);
}

// Measured, us at N x K = 14336 x 4096 | 8192 x 2048 | 2048 x 2048 | 50001 x
// 2048 (weights from HBM):
//   M 1    rows 14.4 | 5.6 | 2.8 | 22.7    frag 15.9 | 6.5 | 3.9 | 22.6
//   M 4    rows 12.4 | 6.9 | 2.9 | 24.1    frag 16.5 | 6.6 | 3.9 | 23.6
//   M 8    rows 22.9 | 11.9 | 4.9 | 47.2   frag 16.8 | 6.6 | 3.9 | 24.8
//   M 16   frag 17.9 | 8.3 | 4.8 | 33.1    mma 19.7 | 11.4 | 10.2 | 30.6
//   M 32   frag 23.7 | 12.4 | 5.7 | 49.6   mma 19.8 | 11.4 | 10.3 | 35.7
//   M 128  mma 27.1 | 14.0 | 11.7 | 49.2
//   M 129  pair 28.3 | 16.2 | 13.6 | 52.5
template <typename E>
cudaError_t matmul_t(const Q8Args &a, cudaStream_t s) {
  if (a.M == 1) return rows_t<E, 1>(a, s);
  if (a.M == 2) return rows_t<E, 2>(a, s);
  if (a.M <= ROWS_MAX) return rows_t<E, 4>(a, s);
  if (a.M <= 8) return frag_t<E, 1>(a, s);
  if (a.M <= 16) return frag_t<E, 2>(a, s);
  if (a.M <= 32 && a.N <= 4096) return frag_mt<E, 4, 1>(a, s);
  return a.M < PAIR_MIN ? mma_t<E>(a, s) : pair_t<E>(a, s);
}

}  // namespace

size_t q8_scratch(int M, int N, int K) {
  (void)N;
  return M < PAIR_MIN ? 0 : ((size_t)M * K * 2 + 255) / 256 * 256;  // a in fp16
}

cudaError_t launch_q8_matmul(const Q8Args &a, cudaStream_t s) {
  const cudaError_t e = a.dtype == TWELL_BF16 ? matmul_t<bf16>(a, s) : matmul_t<float>(a, s);
  prof_mark(KID_Q8_MATMUL, s);
  return e;
}

}  // namespace twell
