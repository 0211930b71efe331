// recur.cu -- gated linear recurrence over packed sequences, and its backward.
//
//   a = sigmoid(gate + bias), c = 1 - a,  h_t = h_{t-1} + c_t (x_t - h_{t-1})
//   G_t = dh_t + a_{t+1} G_{t+1},  dx = c G,  dgate = G (h_{t-1} - x) a c
//
// A row's step is the map h -> (1 - C) h + H; maps compose,
//   (C2, H2) after (C1, H1) = (C1 + C2 - C1 C2, H2 + H1 - C2 H1),
// so time can be cut up.  The share that is taken, C, is kept instead of the one
// that stays: where little is taken at each of many rows, 1 - C would lose it to
// rounding.  A sequence's first row forgets what stood before it ("cut").
//
// HBM bounds it: 3 values an element forward, 5 backward.  To read each value once
// without a wait of CTA on CTA through memory, a cluster of up to 8 CTAs owns a
// slab of channels and goes through all rows: each CTA takes a tile of the rows,
//   a thread composes its rows' steps, a warp its threads' (shuffles), the CTA
//   its warps' (shared memory), the cluster its CTAs' (distributed shared memory),
// and with the state that comes in from the left every thread goes over its rows
// once more, from shared memory, and writes them.  The grouping of the sums follows
// from the sizes alone.  The next tiles' rows are on their way meanwhile.
//
// The backward runs the same over the rows in reverse for G, and forward within a
// tile for h, from the fp32 states that the forward kept every RECUR_KEEP rows: h
// itself is not read (5 values an element instead of 6), and its rounding does not
// enter the gradient.
#include <cooperative_groups.h>

#include "common.cuh"
#include "lm_kernels.h"
#include "vec16.cuh"

namespace cg = cooperative_groups;

namespace twell {

namespace {

constexpr int NT = 256, WARPS = NT / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int STEPS = 4;            // rows of a thread in a tile
constexpr float LOG2E = 1.4426950408889634f;
constexpr float CUT = 2.f;          // a C that stands for: nothing comes through

struct RecurParams {
  const int32_t *starts;
  int B, T, D, len;                 // len: rows of each sequence without starts
  long long ld;
  const float *bias, *h0;
  float *hT, *states;
  const float *dhT;
  float *dbias, *dh0;
  int32_t *status;
};

// The smaller of sigmoid(f) and sigmoid(-f), with the sign of f (from it both follow
// to a few units of their own last place: the larger one is 1 - it).
__device__ __forceinline__ float smaller_gate(float f) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-fabsf(f * LOG2E)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return copysignf(e * r, f);
}
__device__ __forceinline__ float taken(float s) { return signbit(s) ? 1.f + s : s; }       // c
__device__ __forceinline__ float both(float s) { return fabsf(s) - s * s; }                // a c

// What a step (C, H) makes of h.
__device__ __forceinline__ float apply(float C, float H, float h) {
  return C == CUT ? H : fmaf(-C, h, h) + H;
}
// (C, H) := (C2, H2) after it.
__device__ __forceinline__ void then(float &C, float &H, float C2, float H2) {
  H = apply(C2, H2, H);
  C = C == CUT || C2 == CUT ? CUT : fmaf(-C, C2, C) + C2;
}

// Geometry of a slab of CX threads of channels: NT / CX groups of STEPS rows a tile.
template <typename E, int CX>
struct Geo {
  static constexpr int N = VEC16<E>, SLAB = CX * N, GROUPS = NT / CX, R = GROUPS * STEPS;
  static_assert(R % RECUR_KEEP == 0 && RECUR_KEEP % STEPS == 0, "states stand at a group's first row");
};

// Where sequences begin and end in a tile's rows.  With starts, the CTA marks the
// rows in shared memory (three tiles' worth, so that marking needs no barrier of
// its own); without, it follows from the row.
template <int R>
struct Marks {
  int first[3][R], last[3][R];  // the sequence that begins / ends with the row, or -1
  int from[3];                  // the first entry of starts that is not before the tile
};

// The first entry of starts[0 .. B] that is >= row (B + 1: none), by one warp.
__device__ __forceinline__ int first_entry(const RecurParams &p, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = p.B + 1;     // the answer is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const long long at = (long long)lo + (long long)(lane + 1) * step - 1;
    const bool before = at < hi && p.starts[at] < row;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, before));
    const long long top = (long long)lo + (long long)(n + 1) * step - 1;
    lo += n * step;
    if (top < hi) hi = (int)top;
    if (lo > hi) lo = hi;       // (entries that descend)
  }
  return lo;
}

// Marks a tile's rows, by the threads from `tid` on in steps of n.
template <int R>
__device__ __forceinline__ void mark(const RecurParams &p, Marks<R> &m, int buf, int r0, int tid, int n) {
  for (int s = m.from[buf] + tid; s <= p.B; s += n) {
    const int v = p.starts[s];
    if (v > r0 + R || v < r0) break;  // (below: entries that descend)
    if (s < p.B && v < r0 + R && p.starts[s + 1] > v) m.first[buf][v - r0] = s;
    if (s > 0 && v > r0 && p.starts[s - 1] < v) m.last[buf][v - 1 - r0] = s - 1;
  }
}

// Bits of a thread's rows of a tile, and whose they are.
struct RowBits {
  uint32_t first, last, live;
};
template <int R>
__device__ __forceinline__ RowBits row_bits(const RecurParams &p, const Marks<R> &m, int buf, int r0,
                                            int q, int lo, int hi) {
  RowBits b{0, 0, 0};
  const int row = r0 + q * STEPS;
  if (p.starts) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      b.first |= (uint32_t)(m.first[buf][q * STEPS + i] >= 0) << i;
      b.last |= (uint32_t)(m.last[buf][q * STEPS + i] >= 0) << i;
      b.live |= (uint32_t)(row + i >= lo && row + i < hi) << i;
    }
  } else {
    int at = row % p.len;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      b.first |= (uint32_t)(at == 0) << i;
      at = at + 1 == p.len ? 0 : at + 1;
      b.last |= (uint32_t)(at == 0) << i;
      b.live |= (uint32_t)(row + i < p.T) << i;
    }
    b.first &= b.live;
    b.last &= b.live;
  }
  return b;
}
template <int R>
__device__ __forceinline__ int first_of(const RecurParams &p, const Marks<R> &m, int buf, int r0, int k) {
  return p.starts ? m.first[buf][k] : (r0 + k) / p.len;
}
template <int R>
__device__ __forceinline__ int last_of(const RecurParams &p, const Marks<R> &m, int buf, int r0, int k) {
  return p.starts ? m.last[buf][k] : (r0 + k) / p.len;
}

// N values of an fp32 [B][D] matrix (zeros without one).
template <int N>
__device__ __forceinline__ void load_state(const float *v, int s, int D, int d, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 r = v ? *(const float4 *)(v + (size_t)s * D + d + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    f[i] = r.x; f[i + 1] = r.y; f[i + 2] = r.z; f[i + 3] = r.w;
  }
}
template <int N>
__device__ __forceinline__ void store_state(float *v, size_t s, int D, int d, const float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *(float4 *)(v + s * D + d + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}

// Empty sequences pass `from` on to `to` (zeros without one); the slab's channels
// [d0, d1), by the cluster's CTAs.  The first slab checks starts.
__device__ __forceinline__ void empty_sequences(const RecurParams &p, const float *from, float *to,
                                                int d0, int d1, int rank, int C) {
  if (!p.starts) return;
  for (long long s = rank * NT + (int)threadIdx.x; s < p.B; s += C * NT) {
    const int a = p.starts[s], b = p.starts[s + 1];
    if (d0 == 0 && (a < 0 || b > p.T || a > b)) set_status(p.status, TWELL_ERR_INDEX);
    if (a == b && to)
      for (int d = d0; d < d1; d += 4) {
        float f[4];
        load_state(from, (int)s, p.D, d, f);
        store_state(to, s, p.D, d, f);
      }
  }
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// A thread's rows of a tile on their way to shared memory: vector i of a stage's
// matrix k at [(k * STEPS + i) * NT], which the same thread reads back.
template <typename E>
__device__ __forceinline__ void fetch(uint4 *stage, int k, const E *src, long long pitch, int row,
                                      int lo, int hi) {
  const uint64_t once = gather_policy<L2_FIRST>();
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    if (row + i >= lo && row + i < hi)
      copy16_async(stage + (k * STEPS + i) * NT + threadIdx.x, src + (size_t)(row + i) * pitch, once);
}

constexpr int FWD_STAGES = 2, BWD_STAGES = 2;

template <typename E, int CX>
__global__ void __launch_bounds__(NT, 2)
recur_forward_kernel(const E *x, const E *gate, E *h, RecurParams p) {
  pdl_begin();
  using G = Geo<E, CX>;
  constexpr int N = G::N, R = G::R, SLAB = G::SLAB;
  extern __shared__ uint4 stages[];
  __shared__ Marks<R> marks;
  __shared__ float2 part[WARPS][SLAB];               // the warps' steps
  __shared__ float2 total[2][MAX_CLUSTER][SLAB];     // the CTAs' steps
  __shared__ float in[WARPS][SLAB];                  // the state before each warp's rows
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  if (C > 1) cluster_arrive();  // (this CTA runs: its shared memory may be written)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = tid / CX, cx = tid % CX;
  const int d0 = (int)(blockIdx.x / C) * SLAB, d = d0 + cx * N;
  const bool on = d < p.D;
  const int lo = p.starts ? max(0, p.starts[0]) : 0, hi = p.starts ? min(p.T, p.starts[p.B]) : p.T;
  const int tiles = (p.T + R - 1) / R, rounds = (tiles + C - 1) / C;
  auto first_row = [&](int i) { return (int)min((long long)p.T, ((long long)i * C + rank) * R); };
  auto load = [&](int i) {
    if (on && i < rounds) {
      uint4 *st = stages + (i % FWD_STAGES) * 2 * STEPS * NT;
      const int row = first_row(i) + q * STEPS;
      fetch(st, 0, x + d, p.ld, row, lo, hi);
      fetch(st, 1, gate + d, p.ld, row, lo, hi);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < FWD_STAGES - 1; ++i) load(i);
  empty_sequences(p, p.h0, p.hT, d0, min(p.D, d0 + SLAB), rank, C);
  float bias[N];
  load_state(on ? p.bias : nullptr, 0, 0, d, bias);
  if (p.starts) {  // the first tile's marks
    for (int k = tid; k < R; k += NT) marks.first[0][k] = marks.last[0][k] = -1;
    if (warp == 0) {
      const int s = first_entry(p, first_row(0));
      if (lane == 0) marks.from[0] = s;
    }
    __syncthreads();
    mark(p, marks, 0, first_row(0), tid, NT);
    __syncthreads();
  }
  float carry = 0.f;  // the state before the cluster's next rows (threads of the slab)
  if (C > 1) cluster_wait();
  for (int i = 0; i < rounds; ++i) {
    const int r0 = first_row(i), buf = i % 3, next = (i + 1) % 3, row = r0 + q * STEPS;
    const uint4 *st = stages + (i % FWD_STAGES) * 2 * STEPS * NT + tid;
    load(i + FWD_STAGES - 1);
    if (p.starts && i + 1 < rounds) {
      for (int k = tid; k < R; k += NT) marks.first[next][k] = marks.last[next][k] = -1;
      if (warp == WARPS - 1) {
        const int s = first_entry(p, first_row(i + 1));
        if (lane == 0) marks.from[next] = s;
      }
    }
    const RowBits bits = row_bits(p, marks, buf, r0, q, lo, hi);
    asm volatile("cp.async.wait_group %0;" ::"n"(FWD_STAGES - 1) : "memory");
    // this thread's rows as one step
    float c[STEPS][N], Cs[N], Hs[N];
#pragma unroll
    for (int n = 0; n < N; ++n) Cs[n] = Hs[n] = 0.f;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      float xv[N], gv[N];
      unpack(st[k * NT], xv, (E *)nullptr);
      unpack(st[(STEPS + k) * NT], gv, (E *)nullptr);
      const bool live = bits.live >> k & 1, first = bits.first >> k & 1;
      if (first && on) load_state(p.h0, first_of(p, marks, buf, r0, q * STEPS + k), p.D, d, Hs);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        c[k][n] = taken(smaller_gate(gv[n] + bias[n]));
        Hs[n] = live ? fmaf(c[k][n], xv[n] - Hs[n], Hs[n]) : 0.f;
        Cs[n] = first || !live ? CUT : Cs[n] == CUT ? CUT : fmaf(-Cs[n], c[k][n], Cs[n]) + c[k][n];
      }
    }
    // the steps of the warp's groups up to this one, and up to the one before
    float Ce[N], He[N];
#pragma unroll
    for (int o = CX; o < 32; o *= 2) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float C1 = __shfl_up_sync(0xFFFFFFFFu, Cs[n], o), H1 = __shfl_up_sync(0xFFFFFFFFu, Hs[n], o);
        if (lane >= o) {
          then(C1, H1, Cs[n], Hs[n]);
          Cs[n] = C1;
          Hs[n] = H1;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      Ce[n] = __shfl_up_sync(0xFFFFFFFFu, Cs[n], CX);
      He[n] = __shfl_up_sync(0xFFFFFFFFu, Hs[n], CX);
      if (lane < CX) Ce[n] = He[n] = 0.f;
      if (lane >= 32 - CX) part[warp][cx * N + n] = make_float2(Cs[n], Hs[n]);
    }
    __syncthreads();
    if (tid < SLAB) {
      if (C > 1) {  // the CTA's step, to every CTA
        float Ct = 0.f, Ht = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) then(Ct, Ht, part[w][tid].x, part[w][tid].y);
        for (int r = 0; r < C; ++r)
          *cluster.map_shared_rank(&total[i & 1][rank][tid], r) = make_float2(Ct, Ht);
      }
    } else if (p.starts && i + 1 < rounds) {
      mark(p, marks, next, first_row(i + 1), tid - SLAB, NT - SLAB);
    }
    if (C > 1) {
      cluster_arrive();
      cluster_wait();
    }
    if (tid < SLAB) {
      float s = carry;
      if (C > 1)
        for (int r = 0; r < C; ++r) {
          if (r == rank) s = carry;
          const float2 v = total[i & 1][r][tid];
          carry = apply(v.x, v.y, carry);
        }
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        in[w][tid] = s;
        s = apply(part[w][tid].x, part[w][tid].y, s);
      }
      if (C == 1) carry = s;
    }
    __syncthreads();
    // the rows once more, from the state before them
    if (on) {
      float y[N];
#pragma unroll
      for (int n = 0; n < N; ++n) y[n] = apply(Ce[n], He[n], in[warp][cx * N + n]);
      if (p.states && row % RECUR_KEEP == 0 && row < p.T)
        store_state(p.states, row / RECUR_KEEP, p.D, d, y);
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        float xv[N];
        unpack(st[k * NT], xv, (E *)nullptr);
        if (!(bits.live >> k & 1)) continue;
        if (bits.first >> k & 1)
          load_state(p.h0, first_of(p, marks, buf, r0, q * STEPS + k), p.D, d, y);
#pragma unroll
        for (int n = 0; n < N; ++n) y[n] = fmaf(c[k][n], xv[n] - y[n], y[n]);
        *(uint4 *)(h + (size_t)(row + k) * p.D + d) = pack16(y, (E *)nullptr);
        if ((bits.last >> k & 1) && p.hT)
          store_state(p.hT, last_of(p, marks, buf, r0, q * STEPS + k), p.D, d, y);
      }
    }
  }
}

template <typename E, int CX>
__global__ void __launch_bounds__(NT, 2)
recur_backward_kernel(const E *x, const E *gate, const E *dh, E *dx, E *dgate, RecurParams p) {
  pdl_begin();
  using G = Geo<E, CX>;
  constexpr int N = G::N, R = G::R, SLAB = G::SLAB;
  extern __shared__ uint4 stages[];
  __shared__ Marks<R> marks;
  __shared__ float2 partF[WARPS][SLAB], partB[WARPS][SLAB];  // the warps' steps, forward and back
  __shared__ float2 total[2][MAX_CLUSTER][SLAB];             // the CTAs' steps back
  __shared__ float inF[WARPS][SLAB], inB[WARPS][SLAB];       // h before, a G behind each warp's rows
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  if (C > 1) cluster_arrive();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = tid / CX, cx = tid % CX;
  const int d0 = (int)(blockIdx.x / C) * SLAB, d = d0 + cx * N;
  const bool on = d < p.D;
  const int lo = p.starts ? max(0, p.starts[0]) : 0, hi = p.starts ? min(p.T, p.starts[p.B]) : p.T;
  const int tiles = (p.T + R - 1) / R, rounds = (tiles + C - 1) / C;
  // round i: the cluster's tiles from the last on
  auto first_row = [&](int i) {
    return (int)min((long long)p.T, ((long long)(rounds - 1 - i) * C + rank) * R);
  };
  auto load = [&](int i) {
    if (on && i < rounds) {
      uint4 *st = stages + (i % BWD_STAGES) * 3 * STEPS * NT;
      const int row = first_row(i) + q * STEPS;
      fetch(st, 0, x + d, p.ld, row, lo, hi);
      fetch(st, 1, gate + d, p.ld, row, lo, hi);
      fetch(st, 2, dh + d, p.D, row, lo, hi);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < BWD_STAGES - 1; ++i) load(i);
  empty_sequences(p, p.dhT, p.dh0, d0, min(p.D, d0 + SLAB), rank, C);
  float bias[N], db[N];
  load_state(on ? p.bias : nullptr, 0, 0, d, bias);
#pragma unroll
  for (int n = 0; n < N; ++n) db[n] = 0.f;
  if (p.starts) {
    for (int k = tid; k < R; k += NT) marks.first[0][k] = marks.last[0][k] = -1;
    if (warp == 0) {
      const int s = first_entry(p, first_row(0));
      if (lane == 0) marks.from[0] = s;
    }
    __syncthreads();
    mark(p, marks, 0, first_row(0), tid, NT);
    __syncthreads();
  }
  float carry = 0.f;  // a G behind the cluster's next rows (threads of the slab)
  if (C > 1) cluster_wait();
  for (int i = 0; i < rounds; ++i) {
    const int r0 = first_row(i), buf = i % 3, next = (i + 1) % 3, row = r0 + q * STEPS;
    const uint4 *st = stages + (i % BWD_STAGES) * 3 * STEPS * NT + tid;
    load(i + BWD_STAGES - 1);
    if (p.starts && i + 1 < rounds) {
      for (int k = tid; k < R; k += NT) marks.first[next][k] = marks.last[next][k] = -1;
      if (warp == WARPS - 1) {
        const int s = first_entry(p, first_row(i + 1));
        if (lane == 0) marks.from[next] = s;
      }
    }
    // (the state before the tile; where its first row begins a sequence it is not used)
    float before = 0.f;
    const int ch = tid - SLAB;
    if (ch >= 0 && ch < SLAB && d0 + ch < p.D && r0 > 0 && r0 < p.T)
      before = p.states[(size_t)(r0 / RECUR_KEEP) * p.D + d0 + ch];
    const RowBits bits = row_bits(p, marks, buf, r0, q, lo, hi);
    asm volatile("cp.async.wait_group %0;" ::"n"(BWD_STAGES - 1) : "memory");
    float s[STEPS][N], Cf[N], Hf[N], Cb[N], Hb[N];
#pragma unroll
    for (int n = 0; n < N; ++n) Cf[n] = Hf[n] = Cb[n] = Hb[n] = 0.f;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      float xv[N], gv[N];
      unpack(st[k * NT], xv, (E *)nullptr);
      unpack(st[(STEPS + k) * NT], gv, (E *)nullptr);
      const bool live = bits.live >> k & 1, first = bits.first >> k & 1;
      if (first && on) load_state(p.h0, first_of(p, marks, buf, r0, q * STEPS + k), p.D, d, Hf);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        s[k][n] = smaller_gate(gv[n] + bias[n]);
        const float c = taken(s[k][n]);
        Hf[n] = live ? fmaf(c, xv[n] - Hf[n], Hf[n]) : 0.f;
        Cf[n] = first || !live ? CUT : Cf[n] == CUT ? CUT : fmaf(-Cf[n], c, Cf[n]) + c;
      }
    }
#pragma unroll
    for (int k = STEPS - 1; k >= 0; --k) {
      float dv[N];
      unpack(st[(2 * STEPS + k) * NT], dv, (E *)nullptr);
      const bool live = bits.live >> k & 1, last = bits.last >> k & 1;
      if (last && on) load_state(p.dhT, last_of(p, marks, buf, r0, q * STEPS + k), p.D, d, Hb);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float c = taken(s[k][n]), g = dv[n] + Hb[n];
        Hb[n] = live ? fmaf(-c, g, g) : 0.f;
        Cb[n] = last || !live ? CUT : Cb[n] == CUT ? CUT : fmaf(-Cb[n], c, Cb[n]) + c;
      }
    }
#pragma unroll
    for (int o = CX; o < 32; o *= 2) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float C1 = __shfl_up_sync(0xFFFFFFFFu, Cf[n], o), H1 = __shfl_up_sync(0xFFFFFFFFu, Hf[n], o);
        if (lane >= o) {
          then(C1, H1, Cf[n], Hf[n]);
          Cf[n] = C1;
          Hf[n] = H1;
        }
        C1 = __shfl_down_sync(0xFFFFFFFFu, Cb[n], o);
        H1 = __shfl_down_sync(0xFFFFFFFFu, Hb[n], o);
        if (lane + o < 32) {
          then(C1, H1, Cb[n], Hb[n]);
          Cb[n] = C1;
          Hb[n] = H1;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (lane >= 32 - CX) partF[warp][cx * N + n] = make_float2(Cf[n], Hf[n]);
      if (lane < CX) partB[warp][cx * N + n] = make_float2(Cb[n], Hb[n]);
      Cf[n] = __shfl_up_sync(0xFFFFFFFFu, Cf[n], CX);
      Hf[n] = __shfl_up_sync(0xFFFFFFFFu, Hf[n], CX);
      Cb[n] = __shfl_down_sync(0xFFFFFFFFu, Cb[n], CX);
      Hb[n] = __shfl_down_sync(0xFFFFFFFFu, Hb[n], CX);
      if (lane < CX) Cf[n] = Hf[n] = 0.f;
      if (lane >= 32 - CX) Cb[n] = Hb[n] = 0.f;
    }
    __syncthreads();
    if (tid < SLAB) {
      if (C > 1) {
        float Ct = 0.f, Ht = 0.f;
#pragma unroll
        for (int w = WARPS - 1; w >= 0; --w) then(Ct, Ht, partB[w][tid].x, partB[w][tid].y);
        for (int r = 0; r < C; ++r)
          *cluster.map_shared_rank(&total[i & 1][rank][tid], r) = make_float2(Ct, Ht);
      }
    } else if (ch < SLAB) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        inF[w][ch] = before;
        before = apply(partF[w][ch].x, partF[w][ch].y, before);
      }
    } else if (p.starts && i + 1 < rounds) {
      mark(p, marks, next, first_row(i + 1), tid - 2 * SLAB, NT - 2 * SLAB);
    }
    if (C > 1) {
      cluster_arrive();
      cluster_wait();
    }
    if (tid < SLAB) {
      float u = carry;
      if (C > 1)
        for (int r = C - 1; r >= 0; --r) {
          if (r == rank) u = carry;
          const float2 v = total[i & 1][r][tid];
          carry = apply(v.x, v.y, carry);
        }
#pragma unroll
      for (int w = WARPS - 1; w >= 0; --w) {
        inB[w][tid] = u;
        u = apply(partB[w][tid].x, partB[w][tid].y, u);
      }
      if (C == 1) carry = u;
    }
    __syncthreads();
    if (on) {
      float y[N], e[STEPS][N];  // e: (h_{t-1} - x_t) a c
#pragma unroll
      for (int n = 0; n < N; ++n) y[n] = apply(Cf[n], Hf[n], inF[warp][cx * N + n]);
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        float xv[N];
        unpack(st[k * NT], xv, (E *)nullptr);
        if (bits.first >> k & 1)
          load_state(p.h0, first_of(p, marks, buf, r0, q * STEPS + k), p.D, d, y);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const float off = y[n] - xv[n];
          e[k][n] = off * both(s[k][n]);
          y[n] = fmaf(-taken(s[k][n]), off, y[n]);
        }
      }
#pragma unroll
      for (int n = 0; n < N; ++n) y[n] = apply(Cb[n], Hb[n], inB[warp][cx * N + n]);
#pragma unroll
      for (int k = STEPS - 1; k >= 0; --k) {
        float dv[N], gv[N];
        unpack(st[(2 * STEPS + k) * NT], dv, (E *)nullptr);
        if (!(bits.live >> k & 1)) continue;
        if (bits.last >> k & 1)
          load_state(p.dhT, last_of(p, marks, buf, r0, q * STEPS + k), p.D, d, y);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const float c = taken(s[k][n]), g = dv[n] + y[n];
          gv[n] = g * e[k][n];
          db[n] += gv[n];
          dv[n] = c * g;
          y[n] = g - dv[n];
        }
        *(uint4 *)(dx + (size_t)(row + k) * p.ld + d) = pack16(dv, (E *)nullptr);
        *(uint4 *)(dgate + (size_t)(row + k) * p.ld + d) = pack16(gv, (E *)nullptr);
        if ((bits.first >> k & 1) && p.dh0)
          store_state(p.dh0, first_of(p, marks, buf, r0, q * STEPS + k), p.D, d, y);
      }
    }
  }
  if (!p.dbias) return;
  // the bias' gradient: groups of a warp, warps, CTAs, each in order (by way of the
  // totals that the last round does not read)
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int o = 16; o >= CX; o /= 2) db[n] += __shfl_down_sync(0xFFFFFFFFu, db[n], o);
    if (lane < CX) inB[warp][cx * N + n] = db[n];
  }
  __syncthreads();
  float sum = 0.f;
  if (tid < SLAB) {
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += inB[w][tid];
    if (C > 1) cluster.map_shared_rank(&total[rounds & 1][rank][tid], 0)->x = sum;
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    sum = 0.f;
    if (tid < SLAB)
      for (int r = 0; r < C; ++r) sum += total[rounds & 1][r][tid].x;
  }
  if (tid < SLAB && d0 + tid < p.D) p.dbias[d0 + tid] = sum;
}

// Sequences of one row (a decoded token each): a thread for 16 bytes.
template <typename E>
__global__ void __launch_bounds__(NT)
recur_step_kernel(const E *x, const E *gate, E *h, RecurParams p) {
  pdl_begin();
  constexpr int N = VEC16<E>;
  const int per = p.D / N;
  const long long k = (long long)blockIdx.x * NT + threadIdx.x;
  const int row = (int)(k / per), d = (int)(k % per) * N;
  if (row >= p.T) return;
  float xv[N], gv[N], y[N], bias[N];
  unpack(*(const uint4 *)(x + (size_t)row * p.ld + d), xv, (E *)nullptr);
  unpack(*(const uint4 *)(gate + (size_t)row * p.ld + d), gv, (E *)nullptr);
  load_state(p.bias, 0, 0, d, bias);
  load_state(p.h0, row, p.D, d, y);
#pragma unroll
  for (int n = 0; n < N; ++n) y[n] = fmaf(taken(smaller_gate(gv[n] + bias[n])), xv[n] - y[n], y[n]);
  *(uint4 *)(h + (size_t)row * p.D + d) = pack16(y, (E *)nullptr);
  if (p.hT) store_state(p.hT, row, p.D, d, y);
}

RecurParams params_of(const RecurArgs &a) {
  RecurParams p;
  p.starts = a.starts; p.B = a.B; p.T = a.T; p.D = a.D; p.len = a.T / a.B; p.ld = a.ld;
  p.bias = a.bias; p.h0 = a.h0; p.hT = a.hT; p.states = a.states; p.dhT = a.dhT;
  p.dbias = a.dbias; p.dh0 = a.dh0; p.status = a.status;
  return p;
}

// CTAs of a cluster: as many as there are tiles, up to 8, while the grid is less
// than two CTAs an SM.
template <typename E, int CX>
int cluster_of(const RecurArgs &a, int slabs) {
  const int tiles = (a.T + Geo<E, CX>::R - 1) / Geo<E, CX>::R;
  int C = 1;
  while (C < MAX_CLUSTER && C < tiles && slabs * C < 2 * num_sms()) C *= 2;
  return C;
}

template <typename E, int CX>
cudaError_t forward_t(const RecurArgs &a, cudaStream_t s) {
  const int slabs = (a.D + Geo<E, CX>::SLAB - 1) / Geo<E, CX>::SLAB, C = cluster_of<E, CX>(a, slabs);
  constexpr int SMEM = FWD_STAGES * 2 * STEPS * NT * 16;
  auto kern = recur_forward_kernel<E, CX>;
  static const cudaError_t attr =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (attr != cudaSuccess) return attr;
  return launch_clusters(kern, dim3((unsigned)(slabs * C)), dim3(NT), SMEM, C, s, (const E *)a.x,
                         (const E *)a.gate, (E *)a.h, params_of(a));
}

template <typename E, int CX>
cudaError_t backward_t(const RecurArgs &a, cudaStream_t s) {
  const int slabs = (a.D + Geo<E, CX>::SLAB - 1) / Geo<E, CX>::SLAB, C = cluster_of<E, CX>(a, slabs);
  constexpr int SMEM = BWD_STAGES * 3 * STEPS * NT * 16;
  auto kern = recur_backward_kernel<E, CX>;
  static const cudaError_t attr =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (attr != cudaSuccess) return attr;
  return launch_clusters(kern, dim3((unsigned)(slabs * C)), dim3(NT), SMEM, C, s, (const E *)a.x,
                         (const E *)a.gate, (const E *)a.dh, (E *)a.dx, (E *)a.dgate, params_of(a));
}

// Channels of a slab: 128 bytes of a row, or less where the grid would not fill the SMs.
template <typename E>
int threads_across(const RecurArgs &a) {
  const int vecs = a.D / VEC16<E>;
  int cx = 8;
  while (cx > 2 && (vecs + cx - 1) / cx * MAX_CLUSTER < num_sms()) cx /= 2;
  return cx;
}

template <typename E>
cudaError_t forward_e(const RecurArgs &a, cudaStream_t s) {
  if (!a.starts && a.B == a.T) {
    const long long vecs = (long long)a.T * (a.D / VEC16<E>);
    return launch_k(recur_step_kernel<E>, dim3((unsigned)((vecs + NT - 1) / NT)), dim3(NT), 0, s,
                    (const E *)a.x, (const E *)a.gate, (E *)a.h, params_of(a));
  }
  const int cx = threads_across<E>(a);
  return cx == 8 ? forward_t<E, 8>(a, s) : cx == 4 ? forward_t<E, 4>(a, s) : forward_t<E, 2>(a, s);
}

template <typename E>
cudaError_t backward_e(const RecurArgs &a, cudaStream_t s) {
  const int cx = threads_across<E>(a);
  return cx == 8 ? backward_t<E, 8>(a, s) : cx == 4 ? backward_t<E, 4>(a, s) : backward_t<E, 2>(a, s);
}

}  // namespace

cudaError_t launch_recur_forward(const RecurArgs &a, cudaStream_t s) {
  return a.dtype == TWELL_BF16 ? forward_e<bf16>(a, s) : forward_e<float>(a, s);
}

cudaError_t launch_recur_backward(const RecurArgs &a, cudaStream_t s) {
  return a.dtype == TWELL_BF16 ? backward_e<bf16>(a, s) : backward_e<float>(a, s);
}

}  // namespace twell
