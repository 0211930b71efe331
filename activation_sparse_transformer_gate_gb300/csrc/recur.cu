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

constexpr int NT = 128;             // threads of a CTA
constexpr int MAX_CLUSTER = 8;
constexpr int FWD_STEPS = 8, BWD_STEPS = 4;  // rows of a thread in a tile
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

__device__ __forceinline__ float ex2_approx(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}
// c from exp(f), to a few units of its own last place on either side (0 where exp(f)
// has overflowed).
__device__ __forceinline__ float taken(float e) {
  float c;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(1.f + e));
  return c;
}
// exp(f) held below 2^127.5, where c has been flushed to 0 and e c is a number.
__device__ __forceinline__ float ex2_held(float t) {
  float m;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(t), "f"(127.5f));
  return ex2_approx(m);
}

// What a step (C, H) makes of h.  CLEAN: where no step is cut.
template <bool CLEAN = false>
__device__ __forceinline__ float apply(float C, float H, float h) {
  const float r = fmaf(-C, h, h) + H;
  return !CLEAN && C == CUT ? H : r;
}
// (C, H) := (C2, H2) after it.
template <bool CLEAN>
__device__ __forceinline__ void then(float &C, float &H, float C2, float H2) {
  H = apply<CLEAN>(C2, H2, H);
  const float r = fmaf(-C, C2, C) + C2;
  C = !CLEAN && (C == CUT || C2 == CUT) ? CUT : r;
}

// Geometry of a slab of CX threads of channels: NT / CX groups of S rows a tile.
// For the scan over the groups a channel has PARTS threads, lanes of one warp, with
// N consecutive groups each.
template <typename E, int CX, int S>
struct Geo {
  static constexpr int N = VEC16<E>, SLAB = CX * N, GROUPS = NT / CX, R = GROUPS * S;
  static constexpr int PARTS = NT / SLAB, ACROSS = 32 / PARTS;  // a warp's channels in the scan
  static_assert(R % RECUR_KEEP == 0 && RECUR_KEEP % S == 0, "states stand at a group's first row");
  static_assert(PARTS * N == GROUPS && PARTS <= 32, "a warp holds a channel's groups");
  static_assert(SLAB >= 16, "columns are exchanged within 16");
  // Where the step of group q's channel n * CX + cx stands: rows of SLAB pairs, whose
  // columns are exchanged so that neither the threads of the rows (q and cx vary, n
  // does not) nor those of the scan (channels and parts vary) meet in a bank.
  __device__ static __forceinline__ int at(int q, int ch) {
    return q * SLAB + (ch ^ (((q / N * ACROSS) ^ (q % (16 / CX) * CX)) & 15));
  }
};

// Where sequences begin and end in a tile's rows.  With starts, the CTA marks the
// rows in shared memory (three tiles' worth, so that marking needs no barrier of
// its own); without, it follows from the row.
template <int R>
struct Marks {
  uint32_t firsts[3][R / 32], lasts[3][R / 32];  // bits of the rows
  int first[3][R], last[3][R];  // the sequence that begins / ends with a marked row
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

// What has to be done before the barrier that marking stands behind.
template <int R>
__device__ __forceinline__ void begin_marks(const RecurParams &p, Marks<R> &m, int buf, int r0) {
  if (!p.starts) return;
  if (threadIdx.x < R / 32) m.firsts[buf][threadIdx.x] = m.lasts[buf][threadIdx.x] = 0;
  static_assert(R / 32 <= NT, "a word a thread");
  if (threadIdx.x >= NT - 32) {
    const int s = first_entry(p, r0);
    if (threadIdx.x == NT - 1) m.from[buf] = s;
  }
}
// Marks a tile's rows.
template <int R>
__device__ __forceinline__ void mark(const RecurParams &p, Marks<R> &m, int buf, int r0) {
  if (!p.starts) return;
  for (int s = m.from[buf] + (int)threadIdx.x; s <= p.B; s += NT) {
    const int v = p.starts[s], k = v - r0;
    if (v > r0 + R || v < r0) break;  // (below: entries that descend)
    if (s < p.B && k < R && p.starts[s + 1] > v) {
      m.first[buf][k] = s;
      atomicOr(&m.firsts[buf][k / 32], 1u << (k & 31));
    }
    if (s > 0 && k > 0 && p.starts[s - 1] < v) {
      m.last[buf][k - 1] = s - 1;
      atomicOr(&m.lasts[buf][(k - 1) / 32], 1u << ((k - 1) & 31));
    }
  }
}
template <int R>
__device__ __forceinline__ void first_marks(const RecurParams &p, Marks<R> &m, int r0) {
  if (!p.starts) return;
  begin_marks(p, m, 0, r0);
  __syncthreads();
  mark(p, m, 0, r0);
  __syncthreads();
}

// Bits of a thread's S rows of a tile.
struct RowBits {
  uint32_t first, last, live;
};
// Those of rows row .. row + S - 1 that are in [lo, hi).
template <int S>
__device__ __forceinline__ uint32_t live_rows(int row, int lo, int hi) {
  constexpr uint32_t ALL = (1u << S) - 1;
  const int below = min(max(lo - row, 0), S), upto = min(max(hi - row, 0), S);
  return (ALL << below) & ALL & ((1u << upto) - 1);
}
template <int S, int R>
__device__ __forceinline__ RowBits row_bits(const RecurParams &p, const Marks<R> &m, int buf, int row,
                                            int q, uint32_t live) {
  constexpr uint32_t ALL = (1u << S) - 1;
  RowBits b{0, 0, live};
  if (p.starts) {
    const int k = q * S;  // (S divides 32: a thread's rows are of one word)
    b.first = m.firsts[buf][k / 32] >> (k & 31) & ALL;
    b.last = m.lasts[buf][k / 32] >> (k & 31) & ALL;
  } else {
    int at = row % p.len;
    if (at == 0 || at + S >= p.len) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        b.first |= (uint32_t)(at == 0) << i;
        at = at + 1 == p.len ? 0 : at + 1;
        b.last |= (uint32_t)(at == 0) << i;
      }
    }
  }
  b.first &= live;
  b.last &= live;
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

// A thread's rows of a tile on their way to shared memory: row i to slot[i * NT],
// which the same thread reads back.
template <int S, typename E>
__device__ __forceinline__ void fetch(uint4 *slot, const E *src, long long pitch, int row,
                                      uint32_t live) {
  const uint64_t once = gather_policy<L2_FIRST>();
  const E *at = src + (size_t)row * pitch;
#pragma unroll
  for (int i = 0; i < S; ++i, at += pitch)
    if (live >> i & 1) copy16_async(slot + i * NT, at, once);
}

// The scan over a tile's groups, from the tile's first row on (BACK: from its last):
// replaces each group's step in `steps` by the value that reaches the group;
// `exchange` gives what reaches the tile, from the tile's own step.
template <typename G, bool BACK, bool CLEAN, typename F>
__device__ __forceinline__ void scan_groups(float2 *steps, F exchange) {
  constexpr int N = G::N, P = G::PARTS, W = G::ACROSS;
  constexpr uint32_t FULL = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, part = lane / W, ch = (int)(threadIdx.x >> 5) * W + lane % W;
  float2 v[N];
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = steps[G::at(part * N + j, ch)];
  float C = v[BACK ? N - 1 : 0].x, H = v[BACK ? N - 1 : 0].y;
#pragma unroll
  for (int k = 1; k < N; ++k) {
    const int j = BACK ? N - 1 - k : k;
    then<CLEAN>(C, H, v[j].x, v[j].y);
  }
  const int behind = BACK ? P - 1 - part : part;  // parts that come before this one
#pragma unroll
  for (int o = 1; o < P; o *= 2) {
    float C1 = BACK ? __shfl_down_sync(FULL, C, o * W) : __shfl_up_sync(FULL, C, o * W);
    float H1 = BACK ? __shfl_down_sync(FULL, H, o * W) : __shfl_up_sync(FULL, H, o * W);
    if (behind >= o) {
      then<CLEAN>(C1, H1, C, H);
      C = C1;
      H = H1;
    }
  }
  const int whole = (BACK ? 0 : 32 - W) + lane % W;  // the lane that has the tile's step
  float h = exchange(ch, part, __shfl_sync(FULL, C, whole), __shfl_sync(FULL, H, whole));
  const float C1 = BACK ? __shfl_down_sync(FULL, C, W) : __shfl_up_sync(FULL, C, W);
  const float H1 = BACK ? __shfl_down_sync(FULL, H, W) : __shfl_up_sync(FULL, H, W);
  if (behind > 0) h = apply<CLEAN>(C1, H1, h);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int j = BACK ? N - 1 - k : k;
    steps[G::at(part * N + j, ch)].x = h;
    h = apply<CLEAN>(v[j].x, v[j].y, h);
  }
}

// What reaches this CTA's tile, from the cluster's tiles' steps in the order of the
// rows (BACK: against it); `carry` is what reaches the cluster's first one, and then
// the first one of its next round.  Steps of CTAs that the cluster does not have are
// (0, 0).
template <typename G, bool BACK>
__device__ __forceinline__ float exchange_totals(cg::cluster_group &cluster, int n, int rank,
                                                 float2 (*total)[G::SLAB], int ch, int part, float C,
                                                 float H, float &carry) {
  if (n == 1) {
    const float in = carry;
    carry = apply(C, H, carry);
    return in;
  }
  for (int r = part; r < n; r += G::PARTS)
    *cluster.map_shared_rank(&total[rank][ch], r) = make_float2(C, H);
  cluster_arrive();
  cluster_wait();
  float in = carry;
#pragma unroll
  for (int k = 0; k < MAX_CLUSTER; ++k) {
    const int r = BACK ? MAX_CLUSTER - 1 - k : k;
    if (r == rank) in = carry;
    const float2 v = total[r][ch];
    carry = apply(v.x, v.y, carry);
  }
  return in;
}

// Rounds of a cluster's tiles.
struct Rounds {
  int C, rank, R, n;
  __device__ __forceinline__ Rounds(int C_, int rank_, int R_, int T)
      : C(C_), rank(rank_), R(R_), n(((T + R_ - 1) / R_ + C_ - 1) / C_) {}
  // first row of this CTA's tile in the i-th of them (T where it has none)
  __device__ __forceinline__ int row(int i, int T) const {
    return (int)min((long long)T, ((long long)i * C + rank) * R);
  }
};

template <typename E, int CX>
__global__ void __launch_bounds__(NT, 3)
recur_forward_kernel(const E *x, const E *gate, E *h, RecurParams p) {
  pdl_begin();
  using G = Geo<E, CX, FWD_STEPS>;
  constexpr int N = G::N, R = G::R, SLAB = G::SLAB, S = FWD_STEPS;
  constexpr uint32_t ALL = (1u << S) - 1;
  extern __shared__ uint4 stages[];                  // x of two tiles, gates of one
  __shared__ Marks<R> marks;
  __shared__ float2 steps[G::GROUPS * SLAB];         // the groups' steps, then what reaches them
  __shared__ float2 total[2][MAX_CLUSTER][SLAB];     // the CTAs' steps
  // h0 of the last sequence that begins in each thread's rows: hT may be h0, and who
  // comes to that sequence's end first is open (the others end in the same thread)
  __shared__ float4 held[N / 4][NT];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x;
  for (int k = tid; k < 2 * MAX_CLUSTER * SLAB; k += NT) (&total[0][0][0])[k] = make_float2(0.f, 0.f);
  __syncthreads();
  if (C > 1) cluster_arrive();  // (from here on the others may write to this CTA's memory)
  const int q = tid / CX, cx = tid % CX;
  const int d0 = (int)(blockIdx.x / C) * SLAB, d = d0 + cx * N;
  const bool on = d < p.D;
  const int lo = p.starts ? max(0, p.starts[0]) : 0, hi = p.starts ? min(p.T, max(0, p.starts[p.B])) : p.T;
  const Rounds rounds(C, rank, R, p.T);
  uint4 *const xs = stages + tid, *const gs = stages + 2 * S * NT + tid;
  auto live_of = [&](int i) { return live_rows<S>(rounds.row(i, p.T) + q * S, lo, hi); };
  uint32_t live = live_of(0);
  if (on) {
    fetch<S>(xs, x + d, p.ld, rounds.row(0, p.T) + q * S, live);
    fetch<S>(gs, gate + d, p.ld, rounds.row(0, p.T) + q * S, live);
  }
  empty_sequences(p, p.h0, p.hT, d0, min(p.D, d0 + SLAB), rank, C);
  float bias[N];
  load_state(on ? p.bias : nullptr, 0, 0, d, bias);
#pragma unroll
  for (int n = 0; n < N; ++n) bias[n] *= LOG2E;
  first_marks(p, marks, rounds.row(0, p.T));
  float carry = 0.f;  // the state before the cluster's next rows, of the scan's channel
  if (C > 1) cluster_wait();
  for (int i = 0; i < rounds.n; ++i) {
    const int r0 = rounds.row(i, p.T), buf = i % 3, row = r0 + q * S;
    uint4 *const st = xs + (i & 1) * S * NT;
    const bool more = i + 1 < rounds.n;
    const int r1 = more ? rounds.row(i + 1, p.T) : p.T;
    const uint32_t next = more ? live_of(i + 1) : 0, wanted = on ? next : 0;
    asm volatile("cp.async.wait_all;" ::: "memory");
    fetch<S>(xs + (~i & 1) * S * NT, x + d, p.ld, r1 + q * S, wanted);
    if (more) begin_marks(p, marks, (i + 1) % 3, r1);
    const RowBits bits = row_bits<S>(p, marks, buf, row, q, live);
    // this thread's rows as one step
    float c[S][N], Cs[N], Hs[N];
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (k == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) Cs[n] = Hs[n] = 0.f;
      }
      if (bits.first >> k & 1) {
        load_state(on ? p.h0 : nullptr, first_of(p, marks, buf, r0, q * S + k), p.D, d, Hs);
#pragma unroll
        for (int n = 0; n < N; n += 4)
          held[n / 4][tid] = make_float4(Hs[n], Hs[n + 1], Hs[n + 2], Hs[n + 3]);
      }
      float xv[N], gv[N];
      unpack(st[k * NT], xv, (E *)nullptr);
      unpack(gs[k * NT], gv, (E *)nullptr);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        c[k][n] = taken(ex2_approx(fmaf(gv[n], LOG2E, bias[n])));
        Hs[n] = fmaf(c[k][n], xv[n] - Hs[n], Hs[n]);
        Cs[n] = fmaf(-Cs[n], c[k][n], Cs[n]) + c[k][n];
      }
      if (!(live >> k & 1)) {  // (what was not read may be anything)
#pragma unroll
        for (int n = 0; n < N; ++n) Hs[n] = 0.f;
      }
    }
    fetch<S>(gs, gate + d, p.ld, r1 + q * S, wanted);
    const bool cut = bits.first != 0 || live != ALL;
#pragma unroll
    for (int n = 0; n < N; ++n)
      steps[G::at(q, n * CX + cx)] = make_float2(cut ? CUT : Cs[n], Hs[n]);
    const bool cuts = __syncthreads_or(cut);
    if (more) mark(p, marks, (i + 1) % 3, r1);
    auto exchange = [&](int ch, int part, float Ct, float Ht) {
      return exchange_totals<G, false>(cluster, C, rank, total[i & 1], ch, part, Ct, Ht, carry);
    };
    if (cuts) scan_groups<G, false, false>(steps, exchange);
    else scan_groups<G, false, true>(steps, exchange);
    __syncthreads();
    // the rows once more, from the state before them
    if (on) {
      float y[N];
#pragma unroll
      for (int n = 0; n < N; ++n) y[n] = steps[G::at(q, n * CX + cx)].x;
      if (p.states && row % RECUR_KEEP == 0 && row < p.T)
        store_state(p.states, row / RECUR_KEEP, p.D, d, y);
      E *out = h + (size_t)row * p.D + d;
#pragma unroll
      for (int k = 0; k < S; ++k, out += p.D) {
        float xv[N];
        unpack(st[k * NT], xv, (E *)nullptr);
        if (!(live >> k & 1)) continue;
        if (bits.first >> k == 1) {
#pragma unroll
          for (int n = 0; n < N; n += 4) {
            const float4 v = held[n / 4][tid];
            y[n] = v.x; y[n + 1] = v.y; y[n + 2] = v.z; y[n + 3] = v.w;
          }
        } else if (bits.first >> k & 1) {
          load_state(p.h0, first_of(p, marks, buf, r0, q * S + k), p.D, d, y);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) y[n] = fmaf(c[k][n], xv[n] - y[n], y[n]);
        *(uint4 *)out = pack16(y, (E *)nullptr);
        if ((bits.last >> k & 1) && p.hT)
          store_state(p.hT, last_of(p, marks, buf, r0, q * S + k), p.D, d, y);
      }
    }
    live = next;
  }
}

template <typename E, int CX>
__global__ void __launch_bounds__(NT, 3)
recur_backward_kernel(const E *x, const E *gate, const E *dh, E *dx, E *dgate, RecurParams p) {
  pdl_begin();
  using G = Geo<E, CX, BWD_STEPS>;
  constexpr int N = G::N, R = G::R, SLAB = G::SLAB, S = BWD_STEPS;
  constexpr uint32_t ALL = (1u << S) - 1;
  extern __shared__ uint4 stages[];                  // x and dh of two tiles, gates of one
  __shared__ Marks<R> marks;
  __shared__ float2 steps[2][G::GROUPS * SLAB];      // the groups' steps: h forward, a G back
  __shared__ float2 total[2][MAX_CLUSTER][SLAB];     // the CTAs' steps back
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int k = tid; k < 2 * MAX_CLUSTER * SLAB; k += NT) (&total[0][0][0])[k] = make_float2(0.f, 0.f);
  __syncthreads();
  if (C > 1) cluster_arrive();
  const int q = tid / CX, cx = tid % CX;
  const int d0 = (int)(blockIdx.x / C) * SLAB, d = d0 + cx * N;
  const bool on = d < p.D;
  const int lo = p.starts ? max(0, p.starts[0]) : 0, hi = p.starts ? min(p.T, max(0, p.starts[p.B])) : p.T;
  const Rounds rounds(C, rank, R, p.T);
  auto first_row = [&](int i) { return rounds.row(rounds.n - 1 - i, p.T); };  // from the last on
  uint4 *const xs = stages + tid, *const ds = stages + 2 * S * NT + tid,
        *const gs = stages + 4 * S * NT + tid;
  auto live_of = [&](int i) { return live_rows<S>(first_row(i) + q * S, lo, hi); };
  uint32_t live = live_of(0);
  if (on) {
    fetch<S>(xs, x + d, p.ld, first_row(0) + q * S, live);
    fetch<S>(ds, dh + d, p.D, first_row(0) + q * S, live);
    fetch<S>(gs, gate + d, p.ld, first_row(0) + q * S, live);
  }
  empty_sequences(p, p.dhT, p.dh0, d0, min(p.D, d0 + SLAB), rank, C);
  float bias[N], db[N];
  load_state(on ? p.bias : nullptr, 0, 0, d, bias);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    bias[n] *= LOG2E;
    db[n] = 0.f;
  }
  first_marks(p, marks, first_row(0));
  float carry = 0.f;  // a G behind the cluster's next rows, of the scan's channel
  const int sc = warp * G::ACROSS + lane % G::ACROSS, sd = d0 + sc % CX * N + sc / CX;
  if (C > 1) cluster_wait();
  for (int i = 0; i < rounds.n; ++i) {
    const int r0 = first_row(i), buf = i % 3, row = r0 + q * S;
    uint4 *const xt = xs + (i & 1) * S * NT, *const dt = ds + (i & 1) * S * NT;
    const bool more = i + 1 < rounds.n;
    const int r1 = more ? first_row(i + 1) : p.T;
    const uint32_t next = more ? live_of(i + 1) : 0, wanted = on ? next : 0;
    asm volatile("cp.async.wait_all;" ::: "memory");
    fetch<S>(xs + (~i & 1) * S * NT, x + d, p.ld, r1 + q * S, wanted);
    fetch<S>(ds + (~i & 1) * S * NT, dh + d, p.D, r1 + q * S, wanted);
    if (more) begin_marks(p, marks, (i + 1) % 3, r1);
    // (the state before the tile; where its first row begins a sequence it is not used)
    const float before = sd < p.D && r0 > 0 && r0 < p.T
                             ? p.states[(size_t)(r0 / RECUR_KEEP) * p.D + sd] : 0.f;
    const RowBits bits = row_bits<S>(p, marks, buf, row, q, live);
    float e[S][N], Cs[N], Hs[N], c[S][N];
#pragma unroll
    for (int n = 0; n < N; ++n) Cs[n] = Hs[n] = 0.f;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (bits.first >> k & 1)
        load_state(on ? p.h0 : nullptr, first_of(p, marks, buf, r0, q * S + k), p.D, d, Hs);
      float xv[N], gv[N];
      unpack(xt[k * NT], xv, (E *)nullptr);
      unpack(gs[k * NT], gv, (E *)nullptr);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        e[k][n] = ex2_held(fmaf(gv[n], LOG2E, bias[n]));
        c[k][n] = taken(e[k][n]);
        Hs[n] = fmaf(c[k][n], xv[n] - Hs[n], Hs[n]);
        Cs[n] = fmaf(-Cs[n], c[k][n], Cs[n]) + c[k][n];
      }
      if (!(live >> k & 1)) {
#pragma unroll
        for (int n = 0; n < N; ++n) Hs[n] = 0.f;
      }
    }
    fetch<S>(gs, gate + d, p.ld, r1 + q * S, wanted);
    const bool gap = live != ALL, cutF = gap || bits.first, cutB = gap || bits.last;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      steps[0][G::at(q, n * CX + cx)] = make_float2(cutF ? CUT : Cs[n], Hs[n]);
      Hs[n] = 0.f;
    }
#pragma unroll
    for (int k = S - 1; k >= 0; --k) {
      if (bits.last >> k & 1)
        load_state(on ? p.dhT : nullptr, last_of(p, marks, buf, r0, q * S + k), p.D, d, Hs);
      float dv[N];
      unpack(dt[k * NT], dv, (E *)nullptr);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float g = dv[n] + Hs[n];
        Hs[n] = fmaf(-c[k][n], g, g);
      }
      if (!(live >> k & 1)) {
#pragma unroll
        for (int n = 0; n < N; ++n) Hs[n] = 0.f;
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
      steps[1][G::at(q, n * CX + cx)] = make_float2(cutB ? CUT : Cs[n], Hs[n]);
    const bool cuts = __syncthreads_or(cutF || cutB);
    if (more) mark(p, marks, (i + 1) % 3, r1);
    auto forward = [&](int, int, float, float) { return before; };
    auto exchange = [&](int ch, int part, float Ct, float Ht) {
      return exchange_totals<G, true>(cluster, C, rank, total[i & 1], ch, part, Ct, Ht, carry);
    };
    if (cuts) {
      scan_groups<G, false, false>(steps[0], forward);
      scan_groups<G, true, false>(steps[1], exchange);
    } else {
      scan_groups<G, false, true>(steps[0], forward);
      scan_groups<G, true, true>(steps[1], exchange);
    }
    __syncthreads();
    if (on) {
      float y[N];
#pragma unroll
      for (int n = 0; n < N; ++n) y[n] = steps[0][G::at(q, n * CX + cx)].x;
      // e := (h_{t-1} - x_t) a c
#pragma unroll
      for (int k = 0; k < S; ++k) {
        if (bits.first >> k & 1)
          load_state(p.h0, first_of(p, marks, buf, r0, q * S + k), p.D, d, y);
        float xv[N];
        unpack(xt[k * NT], xv, (E *)nullptr);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const float took = (y[n] - xv[n]) * c[k][n];
          y[n] -= took;
          e[k][n] = took * (e[k][n] * c[k][n]);
        }
      }
#pragma unroll
      for (int n = 0; n < N; ++n) y[n] = steps[1][G::at(q, n * CX + cx)].x;
      E *px = dx + (size_t)row * p.ld + d, *pg = dgate + (size_t)row * p.ld + d;
#pragma unroll
      for (int k = S - 1; k >= 0; --k) {
        if (!(live >> k & 1)) continue;
        if (bits.last >> k & 1)
          load_state(p.dhT, last_of(p, marks, buf, r0, q * S + k), p.D, d, y);
        float dv[N], gv[N];
        unpack(dt[k * NT], dv, (E *)nullptr);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const float g = dv[n] + y[n];
          gv[n] = g * e[k][n];
          db[n] += gv[n];
          dv[n] = c[k][n] * g;
          y[n] = g - dv[n];
        }
        *(uint4 *)(px + k * p.ld) = pack16(dv, (E *)nullptr);
        *(uint4 *)(pg + k * p.ld) = pack16(gv, (E *)nullptr);
        if ((bits.first >> k & 1) && p.dh0)
          store_state(p.dh0, first_of(p, marks, buf, r0, q * S + k), p.D, d, y);
      }
    }
    live = next;
  }
  if (!p.dbias) return;
  // the bias' gradient: groups of a warp, warps, CTAs, each in order (by way of the
  // totals that the last round does not read)
  __shared__ float warps[NT / 32][SLAB];
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int o = 16; o >= CX; o /= 2) db[n] += __shfl_down_sync(0xFFFFFFFFu, db[n], o);
    if (lane < CX) warps[warp][cx * N + n] = db[n];
  }
  __syncthreads();
  float sum = 0.f;
  if (tid < SLAB) {
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) sum += warps[w][tid];
    if (C > 1) cluster.map_shared_rank(&total[rounds.n & 1][rank][tid], 0)->x = sum;
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    sum = 0.f;
    if (tid < SLAB)
      for (int r = 0; r < C; ++r) sum += total[rounds.n & 1][r][tid].x;
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
  for (int n = 0; n < N; ++n) {
    const float c = taken(ex2_approx(fmaf(gv[n], LOG2E, bias[n] * LOG2E)));
    y[n] = fmaf(c, xv[n] - y[n], y[n]);
  }
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

// Clusters of C CTAs of a kernel that are resident at once (0: cannot be told).
template <typename K>
int resident_clusters(K kern, size_t smem, int C) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

// A kernel's clusters: as many CTAs as there are tiles, while all of them are
// resident at once.
template <typename K>
struct Shape {
  cudaError_t attr;
  int fit[MAX_CLUSTER + 1];  // clusters that are resident, by their CTAs
  Shape(K kern, size_t smem)
      : attr(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) {
    for (int C = 1; C <= MAX_CLUSTER; ++C)
      fit[C] = attr == cudaSuccess ? resident_clusters(kern, smem, C) : 0;
  }
  int cluster(int slabs, int tiles) const {
    int C = 1;
    for (int k = 2; k <= MAX_CLUSTER && k <= tiles; ++k)
      if (fit[k] >= slabs) C = k;
    if (const char *e = getenv("RECUR_CL")) C = min(tiles, atoi(e));
    return C;
  }
};

template <typename E, int CX>
cudaError_t forward_t(const RecurArgs &a, cudaStream_t s) {
  using G = Geo<E, CX, FWD_STEPS>;
  constexpr int SMEM = 3 * FWD_STEPS * NT * 16;
  auto kern = recur_forward_kernel<E, CX>;
  static const Shape<decltype(kern)> shape(kern, SMEM);
  if (shape.attr != cudaSuccess) return shape.attr;
  const int slabs = (a.D + G::SLAB - 1) / G::SLAB, C = shape.cluster(slabs, (a.T + G::R - 1) / G::R);
  return launch_clusters(kern, dim3((unsigned)(slabs * C)), dim3(NT), SMEM, C, s, (const E *)a.x,
                         (const E *)a.gate, (E *)a.h, params_of(a));
}

template <typename E, int CX>
cudaError_t backward_t(const RecurArgs &a, cudaStream_t s) {
  using G = Geo<E, CX, BWD_STEPS>;
  constexpr int SMEM = 5 * BWD_STEPS * NT * 16;
  auto kern = recur_backward_kernel<E, CX>;
  static const Shape<decltype(kern)> shape(kern, SMEM);
  if (shape.attr != cudaSuccess) return shape.attr;
  const int slabs = (a.D + G::SLAB - 1) / G::SLAB, C = shape.cluster(slabs, (a.T + G::R - 1) / G::R);
  return launch_clusters(kern, dim3((unsigned)(slabs * C)), dim3(NT), SMEM, C, s, (const E *)a.x,
                         (const E *)a.gate, (const E *)a.dh, (E *)a.dx, (E *)a.dgate, params_of(a));
}

// Channels of a slab: 128 bytes of a row, or less where the grid would not fill the SMs.
template <typename E>
int threads_across(const RecurArgs &a) {
  const int vecs = a.D / VEC16<E>;
  int cx = 8;
  const int least = 16 / VEC16<E>;  // (a slab has 16 channels at least)
  while (cx > least && (vecs + cx - 1) / cx * MAX_CLUSTER < num_sms()) cx /= 2;
  if (const char *e = getenv("RECUR_CX")) cx = atoi(e);
  if (cx < least) cx = least;
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
  if constexpr (VEC16<E> == 8)
    if (cx == 2) return forward_t<E, 2>(a, s);
  return cx == 8 ? forward_t<E, 8>(a, s) : forward_t<E, 4>(a, s);
}

template <typename E>
cudaError_t backward_e(const RecurArgs &a, cudaStream_t s) {
  const int cx = threads_across<E>(a);
  if constexpr (VEC16<E> == 8)
    if (cx == 2) return backward_t<E, 2>(a, s);
  return cx == 8 ? backward_t<E, 8>(a, s) : backward_t<E, 4>(a, s);
}

}  // namespace

cudaError_t launch_recur_forward(const RecurArgs &a, cudaStream_t s) {
  return a.dtype == TWELL_BF16 ? forward_e<bf16>(a, s) : forward_e<float>(a, s);
}

cudaError_t launch_recur_backward(const RecurArgs &a, cudaStream_t s) {
  return a.dtype == TWELL_BF16 ? backward_e<bf16>(a, s) : backward_e<float>(a, s);
}

}  // namespace twell
