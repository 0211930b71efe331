// recur.cu -- gated linear recurrence over packed sequences, and its backward.
//
//   a = sigmoid(gate + bias), c = 1 - a,  h_t = h_{t-1} + c_t (x_t - h_{t-1})
//   G_t = dh_t + a_{t+1} G_{t+1},  dx = c G,  dgate = G (h_{t-1} - x) a c
//
// A row's step is the map h -> A h + H; maps compose,
//   (A2, H2) after (A1, H1) = (A1 A2, H2 + A2 H1),
// so time can be cut up.  Of the share that stays, A, and the one that is taken, 1 - A, the
// smaller is kept: where little is taken at each of many rows, A would lose it to rounding;
// where a gate closes behind a large state, 1 - A would leave that state's rounding in the
// place of what stays of it.  A row's own gate likewise: it goes by c, of which h + c (x - h)
// is one fma, and by a below 2^-6, from where on 1 - c has not the bits that a needs; only
// tiles with such a gate look for it.  A sequence's first row forgets what stood before it
// ("cut").
//
// To read each value once without a wait of CTA on CTA through memory, a cluster of
// up to 16 CTAs owns a slab of channels and goes through all rows in rounds.  A warp
// has 16 channels, or 8, and works by itself (lanes: 2 across and 16 groups of rows,
// or 1 and 32; fp32 has 8 channels on 2 lanes): its tile of a round is 8 rows a group
// (a backward of 16 channels, or of few rows: 4), of which
//   a lane composes its rows' steps, the warp its groups' (shared memory), the cluster
//   its CTAs' (asynchronous stores to distributed shared memory, which an mbarrier
//   counts),
// and with the state that comes in from the left the lanes go over their rows once
// more, from shared memory and registers, and write them.  While a tile's step is on its
// way to the other CTAs, the SM's other CTAs work.  The grouping of the sums follows from
// the sizes and the device.
//
// The backward runs the same over the rows in reverse for G, and forward within a
// tile for h, from the fp32 states that the forward kept every RECUR_KEEP rows: h
// itself is not read (5 values an element instead of 6), and its rounding does not
// enter the gradient.
//
// HBM would bound it (3 values an element forward, 5 backward: 60 and 101 us at 16384 x
// 4096 bf16, which take 81 and 150).  What bounds it is latency, and next the issue slots (41
// and 45%): the gates stay in registers from one pass over a tile to the other, which leaves
// room for 12 warps an SM (8 with 8 rows of bf16 a group and fewer clusters), and a round has
// its fixed part (two scans, the exchange).  Measured on the way: CTAs in step with barriers,
// 150 and 430 us; warps by themselves, 120 and 187; two tiles at a time, one of them on its
// way to the other CTAs, 107 and 186; two channels an instruction, 102 and 183; rows copied
// in whole lines, 95 and 176; tiles copied as boxes of a tensor, 88 and 167; one tile at a
// time again, with the registers spent on more warps and on longer tiles, 84 and 158; copies on
// their way for a whole round, 84 and 142; the smaller share at every joint, 81 and 151; 4 rows
// a group and a third CTA in the backward, 81 and 150 (of 65 sequences 105 and 208, before 104
// and 248).
// Gates computed again in the second pass (24 warps an SM, a round's inputs from L2): 120
// and 258.  Rows copied one by one in bulk: 233 and 251 (32 cycles of the SM each).  One
// body for all tiles, with branches at the rows where sequences begin: 93 and 217; with
// loops over the rows for the tiles that have such: 88 and 170.
#include <cooperative_groups.h>
#include <limits.h>

#include <type_traits>

#include "common.cuh"
#include "lm_kernels.h"
#include "tcgen05.cuh"
#include "vec16.cuh"

namespace cg = cooperative_groups;

namespace twell {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int FEW = 128;            // entries of starts that a CTA keeps at hand
constexpr float CUT = 2.f;          // an m, or A, that stands for: nothing comes through
constexpr float NOTHING = -0.f;     // the m of a step that takes nothing

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
__device__ __forceinline__ float rcp_approx(float t) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

// Pairs of channels: additions, products and fmas of two in one instruction.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 less2(float2 a, float2 b) { return fma2(b, both(-1.f), a); }  // a - b

// A gate as m: -c, or below t = OPEN a, to a few units of its own last place on either side
// (-0: all stays; 0: nothing does).  From OPEN on c's 3 units are 2^-16 of a at most.  What a
// gate gives does not depend on what else is in its tile.
constexpr float OPEN = -6.f;
template <bool CLOSED>
__device__ __forceinline__ float2 gate_of(float2 t, float2 e) {  // t = f log2(e), e = exp(f)
  const float2 u = fma2(e, both(-1.f), both(-1.f));
  float2 m = make_float2(rcp_approx(u.x), rcp_approx(u.y));
  if (CLOSED) {
    if (t.x < OPEN) m.x = e.x * -m.x;
    if (t.y < OPEN) m.y = e.y * -m.y;
  }
  return m;
}
__device__ __forceinline__ float2 exp2_of(float2 t) { return make_float2(ex2_approx(t.x), ex2_approx(t.y)); }
// exp(f) held below 2^127.5, where c has been flushed to 0 and e c is a number.
__device__ __forceinline__ float2 exp2_held(float2 t) {
  float2 m;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m.x) : "f"(t.x), "f"(127.5f));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m.y) : "f"(t.y), "f"(127.5f));
  return exp2_of(m);
}
// a c, where a = e c has all its bits.
template <bool CLOSED>
__device__ __forceinline__ float2 both_shares(float2 t, float2 e, float2 m) {
  float2 r = mul2(mul2(e, m), m);
  if (CLOSED) {
    if (t.x < OPEN) r.x = fmaf(-m.x, m.x, m.x);
    if (t.y < OPEN) r.y = fmaf(-m.y, m.y, m.y);
  }
  return r;
}
__device__ __forceinline__ bool is_c(float m) { return __float_as_int(m) < 0; }
// a where m is -c, else b.
__device__ __forceinline__ float2 pick(float2 m, float2 a, float2 b) {
  return make_float2(is_c(m.x) ? a.x : b.x, is_c(m.y) ? a.y : b.y);
}
// a v, and -c v (CLOSED: m may be either share, else it is -c).
template <bool CLOSED>
__device__ __forceinline__ float2 kept(float2 m, float2 v) {
  return fma2(m, v, CLOSED ? pick(m, v, both(0.f)) : v);
}
template <bool CLOSED>
__device__ __forceinline__ float2 minus_taken(float2 m, float2 v) {
  return CLOSED ? fma2(m, v, pick(m, both(-0.f), make_float2(-v.x, -v.y))) : mul2(m, v);
}
// h + c (x - h), or x + a (h - x); off = h - x.
template <bool CLOSED>
__device__ __forceinline__ float2 row_step(float2 m, float2 x, float2 h, float2 off) {
  return fma2(m, off, CLOSED ? pick(m, h, x) : h);
}
// The lower of two gates, in each place of 16 bytes.
__device__ __forceinline__ uint32_t lower2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2(*(const __nv_bfloat162 *)&a, *(const __nv_bfloat162 *)&b);
  return *(const uint32_t *)&r;
}
__device__ __forceinline__ uint4 lower(const uint4 &a, const uint4 &b, bf16 *) {
  return make_uint4(lower2(a.x, b.x), lower2(a.y, b.y), lower2(a.z, b.z), lower2(a.w, b.w));
}
__device__ __forceinline__ uint32_t lower1(uint32_t a, uint32_t b) {
  return __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint4 lower(const uint4 &a, const uint4 &b, float *) {
  return make_uint4(lower1(a.x, b.x), lower1(a.y, b.y), lower1(a.z, b.z), lower1(a.w, b.w));
}

// 16 bytes of a row as pairs, and back (SIGN: negated).
__device__ __forceinline__ void pairs(const uint4 &u, float2 (&f)[4], bf16 *) {
  f[0] = make_float2(bf_lo(u.x), bf_hi(u.x)); f[1] = make_float2(bf_lo(u.y), bf_hi(u.y));
  f[2] = make_float2(bf_lo(u.z), bf_hi(u.z)); f[3] = make_float2(bf_lo(u.w), bf_hi(u.w));
}
__device__ __forceinline__ void pairs(const uint4 &u, float2 (&f)[2], float *) {
  f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
}
template <bool NEGATED = false>
__device__ __forceinline__ uint4 packed(const float2 (&f)[4], bf16 *) {
  const uint32_t s = NEGATED ? 0x80008000u : 0u;
  return make_uint4(pack_bf2(f[0].x, f[0].y) ^ s, pack_bf2(f[1].x, f[1].y) ^ s,
                    pack_bf2(f[2].x, f[2].y) ^ s, pack_bf2(f[3].x, f[3].y) ^ s);
}
template <bool NEGATED = false>
__device__ __forceinline__ uint4 packed(const float2 (&f)[2], float *) {
  const uint32_t s = NEGATED ? 0x80000000u : 0u;
  return make_uint4(__float_as_uint(f[0].x) ^ s, __float_as_uint(f[0].y) ^ s,
                    __float_as_uint(f[1].x) ^ s, __float_as_uint(f[1].y) ^ s);
}

// What a step stands as in the scan over a tile's groups: m, as a gate does, where the tile's
// own step is asked for (the products of one tile after the other are long); A where it ends
// with the tile.
enum Share { AS_M, AS_A };
// The share that stays (CUT: CUT).
template <Share AS = AS_M>
__device__ __forceinline__ float stays(float v) { return AS == AS_M && is_c(v) ? 1.f + v : v; }
// The m of a share that stays, n: minus what is taken.
__device__ __forceinline__ float smaller(float A, float n) { return A > 0.75f ? n : A; }
// What a step (A, H) makes of h.  CLEAN: where no step is cut.
template <bool CLEAN = false>
__device__ __forceinline__ float apply(float A, float H, float h) {
  const float r = fmaf(A, h, H);
  return !CLEAN && A == CUT ? H : r;
}
// Steps on the way to one: A is what stays, n minus what is taken, each to its own last
// place; n only where all of them are -c (it is asked for where little is taken).
template <Share AS, bool CLEAN>
struct Joint {
  float A, n, H;
  __device__ __forceinline__ Joint(float v, float H_) : A(stays<AS>(v)), n(v), H(H_) {}
  // (v, H) after it
  __device__ __forceinline__ void then(float v, float H2) {
    const float A2 = stays<AS>(v);
    H = apply<CLEAN>(A2, H2, H);
    const bool cut = !CLEAN && (A == CUT || A2 == CUT);
    n = cut ? CUT : fmaf(v, A, n);
    A = cut ? CUT : A2 * A;
  }
  __device__ __forceinline__ float v() const { return AS == AS_M ? smaller(A, n) : A; }
};

// A warp's slab: 16 channels, or 8 (16 or 32 bytes of a row), as CX lanes across; GROUPS
// of lanes take S rows of a tile each.  In the scan over the groups a channel has PARTS
// lanes with N consecutive groups each.
template <typename E, int SLAB_, int S_, int CLUSTER_>
struct Geo {
  static constexpr int N = VEC16<E>, SLAB = SLAB_, CX = SLAB / N, GROUPS = 32 / CX, S = S_, R = GROUPS * S;
  static constexpr int PARTS = 32 / SLAB, ACROSS = SLAB;
  static constexpr int CLUSTER = CLUSTER_;  // CTAs at most
  static constexpr uint32_t ALL = (1u << S) - 1;
  static_assert(R % RECUR_KEEP == 0 && RECUR_KEEP % S == 0, "states stand at a group's first row");
  static_assert(PARTS * N == GROUPS && 32 % S == 0, "lanes hold a channel's groups");
  static_assert(CX == 1 || CX == 2, "see at and the slots");
  // Where the step of group q's channel n * CX + cx stands: rows of SLAB pairs, whose
  // columns are exchanged so that lanes that differ in q and cx do not meet in a bank
  // (nor do those of the scan, which differ in channel and part).
  __device__ static __forceinline__ int at(int q, int ch) {
    const int row = SLAB == 8 ? q ^ (q / N & 1) : q, swap = SLAB == 8 ? row >> 1 : row;
    return row * SLAB + (ch ^ swap % (SLAB / CX) * CX);
  }
};
template <typename E, int SLAB, int CLUSTER> using Fwd = Geo<E, SLAB, 8, CLUSTER>;
template <typename E, int SLAB, int S, int CLUSTER> using Bwd = Geo<E, SLAB, S, CLUSTER>;
constexpr int WARPS = 4;  // a CTA's

// Where sequences begin and end in a warp's tile, by rows.  (Without starts it
// follows from the row.)
template <typename G>
struct Marks {
  static constexpr int R = G::R;
  // (the longest tiles leave no room for more)
  using Index = typename std::conditional<R == 256, uint16_t, int32_t>::type;
  uint32_t firsts[R / 32], lasts[R / 32];  // bits of the rows
  Index first[R], last[R];                 // the sequence that begins / ends with a marked row
};
constexpr int MAX_SHORT_B = 65536;

// The first entry of starts[0 .. B] that is >= row (B + 1: none), by one warp.
__device__ __forceinline__ int first_entry(const int32_t *starts, int B, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B + 1;     // the answer is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const long long at = (long long)lo + (long long)(lane + 1) * step - 1;
    const bool before = at < hi && starts[at] < row;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, before));
    const long long top = (long long)lo + (long long)(n + 1) * step - 1;
    lo += n * step;
    if (top < hi) hi = (int)top;
    if (lo > hi) lo = hi;       // (entries that descend)
  }
  return lo;
}

// An open interval of rows that no entry of starts lies in.
struct Gap {
  int lo = INT_MAX, hi = INT_MIN;
};

// Marks a tile's rows; returns whether there are any.  Most tiles lie within a gap
// that is known already, and cost no look at starts.
template <typename G>
__device__ __forceinline__ bool mark(const int32_t *starts, int B, Marks<G> &m, Gap &gap, int r0) {
  constexpr int R = G::R;
  if (gap.lo < r0 && gap.hi > r0 + R) return false;
  const int lane = threadIdx.x & 31;
  const int from = first_entry(starts, B, r0);
  gap.lo = from > 0 ? starts[from - 1] : INT_MIN;
  gap.hi = from <= B ? starts[from] : INT_MAX;
  __syncwarp();  // (the last tile's marks have been read)
  if (lane < R / 32) m.firsts[lane] = m.lasts[lane] = 0;
  __syncwarp();
  for (int s = from + lane; s <= B; s += 32) {
    const int v = starts[s], k = v - r0;
    if (v > r0 + R || v < r0) break;  // (below: entries that descend)
    if (s < B && k < R && starts[s + 1] > v) {
      m.first[k] = (typename Marks<G>::Index)s;
      atomicOr(&m.firsts[k / 32], 1u << (k & 31));
    }
    if (s > 0 && k > 0 && starts[s - 1] < v) {
      m.last[k - 1] = (typename Marks<G>::Index)(s - 1);
      atomicOr(&m.lasts[(k - 1) / 32], 1u << ((k - 1) & 31));
    }
  }
  __syncwarp();
  return true;
}

// Bits of a thread's S rows of a tile.
struct RowBits {
  uint32_t first, last, live;
  uint32_t any_first, any_last;  // of the warp's lanes (a row that none has costs little)
};
// Those of rows row .. row + S - 1 that are in [lo, hi).
template <int S>
__device__ __forceinline__ uint32_t live_rows(int row, int lo, int hi) {
  constexpr uint32_t ALL = (1u << S) - 1;
  if (row >= lo && row + S <= hi) return ALL;
  const int below = min(max(lo - row, 0), S), upto = min(max(hi - row, 0), S);
  return (ALL << below) & ALL & ((1u << upto) - 1);
}
template <typename G>
__device__ __forceinline__ RowBits row_bits(const RecurParams &p, const int32_t *starts, Marks<G> &m,
                                            Gap &gap, int r0, int q, uint32_t live) {
  constexpr int S = G::S;
  constexpr uint32_t ALL = (1u << S) - 1;
  RowBits b{0, 0, live, 0, 0};
  if (p.starts) {
    if (mark(starts, p.B, m, gap, r0)) {
      const int k = q * S;  // (S divides 32: a lane's rows are of one word)
      b.first = m.firsts[k / 32] >> (k & 31) & ALL;
      b.last = m.lasts[k / 32] >> (k & 31) & ALL;
    }
  } else if (p.len < p.T) {
    int at = (r0 + q * S) % p.len;
    if (at == 0 || at + S >= p.len) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        b.first |= (uint32_t)(at == 0) << i;
        at = at + 1 == p.len ? 0 : at + 1;
        b.last |= (uint32_t)(at == 0) << i;
      }
    }
  } else {
    const int row = r0 + q * S;
    b.first = row == 0;
    if (row < p.T && row + S >= p.T) b.last = 1u << (p.T - 1 - row);
  }
  b.first &= live;
  b.last &= live;
  b.any_first = __reduce_or_sync(0xFFFFFFFFu, b.first);
  b.any_last = __reduce_or_sync(0xFFFFFFFFu, b.last);
  return b;
}
// Whether no sequence begins or ends in the tile from r0 on and all of its rows are some
// sequence's, as far as can be told without a look at starts.
template <int R>
__device__ __forceinline__ bool plain_tile(const RecurParams &p, const Gap &gap, int r0, int lo, int hi) {
  if (!p.starts || r0 < lo || r0 + R > hi) return false;
  return gap.lo < r0 && gap.hi > r0 + R;
}
template <typename G>
__device__ __forceinline__ int first_of(const RecurParams &p, const Marks<G> &m, int r0, int k) {
  return p.starts ? m.first[k] : (r0 + k) / p.len;
}
template <typename G>
__device__ __forceinline__ int last_of(const RecurParams &p, const Marks<G> &m, int r0, int k) {
  return p.starts ? m.last[k] : (r0 + k) / p.len;
}

// M pairs of an fp32 [B][D] matrix (zeros without one).
template <int M>
__device__ __forceinline__ void load_state(const float *v, size_t s, int D, int d, float2 (&f)[M]) {
#pragma unroll
  for (int i = 0; i < M; i += 2) {
    const float4 r = v ? *(const float4 *)(v + s * D + d + 2 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
    f[i] = make_float2(r.x, r.y);
    f[i + 1] = make_float2(r.z, r.w);
  }
}
template <int M>
__device__ __forceinline__ void store_state(float *v, size_t s, int D, int d, const float2 (&f)[M]) {
#pragma unroll
  for (int i = 0; i < M; i += 2)
    *(float4 *)(v + s * D + d + 2 * i) = make_float4(f[i].x, f[i].y, f[i + 1].x, f[i + 1].y);
}

// Empty sequences pass `from` on to `to` (zeros without one): the slab's channels from
// d0 on, by the warps of the cluster's CTAs.  The first slab checks starts.
__device__ __forceinline__ void empty_sequences(const RecurParams &p, const float *from, float *to,
                                                int d0, int d1, int rank, int C) {
  if (!p.starts) return;
  for (long long s = rank * 32 + (int)(threadIdx.x & 31); s < p.B; s += C * 32) {
    const int a = p.starts[s], b = p.starts[s + 1];
    if (d0 == 0 && (a < 0 || b > p.T || a > b)) set_status(p.status, TWELL_ERR_INDEX);
    if (a == b && to)
      for (int d = d0; d < d1; d += 4) {
        float2 f[2];
        load_state(from, s, p.D, d, f);
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

// All warps of the CTA, wherever each of them stands.
__device__ __forceinline__ void cta_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
}

// A CTA's tile of one matrix in shared memory, the channels of its warps, as the copy of
// a tensor's box leaves it: 64 or 128 bytes of a row, whose 16-byte chunks are exchanged
// by the address; the k-th rows of all groups stand together.
template <typename G>
struct alignas(1024) Slot {
  static constexpr int CH = WARPS * G::CX;  // chunks of a row
  uint4 v[G::R * CH];
  static_assert(G::GROUPS % 8 == 0, "a chunk's place follows from q, not from k");
  __device__ static __forceinline__ int at(int q, int k, int chunk) {
    return (k * G::GROUPS + q) * CH + (chunk ^ (CH == 8 ? q & 7 : q >> 1 & 3));
  }
  // A lane's group: eight lanes in a row read one row of 8 / CX groups at once, which are
  // those that do not meet in a bank.
  __device__ static __forceinline__ int group(int g) {
    return G::CX == 1 ? g : (g & 8) | (g << 1 & 6) | (g >> 2 & 1);
  }
};

// The matrices of a call as tensors of (channel, group of S rows, row of the group).
// What T leaves behind the last whole group is not a part of them.
struct Maps {
  CUtensorMap x, gate, dh;
};

// Copies a tile from row r0 on, by one thread.
template <typename G>
__device__ __forceinline__ void fetch(Slot<G> &slot, const CUtensorMap &map, int r0, int d0,
                                      uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(slot.v)),
      "l"((uint64_t)&map), "r"(d0), "r"(r0 / G::S), "r"(0), "r"(bar), "l"(gather_policy<L2_FIRST>())
      : "memory");
}

// starts, in shared memory where there are few (from the CTA's next barrier on).
__device__ __forceinline__ const int32_t *keep_starts(const RecurParams &p, int32_t *few) {
  if (!p.starts || p.B >= FEW) return p.starts;
  for (int k = threadIdx.x; k <= p.B; k += 32 * WARPS) few[k] = p.starts[k];
  return few;
}

// The rows of a tile's last group where T cuts it, a warp's channels of them.
template <typename G, typename E>
__device__ __forceinline__ void fetch_rest(Slot<G> &slot, const E *src, long long pitch, int r0,
                                           int T, int d0, int D) {
  const int lane = threadIdx.x & 31, k = lane / G::CX, cx = lane % G::CX, rest = T % G::S;
  const int d = d0 + cx * G::N, whole = T - rest;
  if (k < rest && d < D)
    slot.v[Slot<G>::at((whole - r0) / G::S, k, (threadIdx.x >> 5) * G::CX + cx)] =
        *(const uint4 *)(src + (size_t)(whole + k) * pitch + d);
}

// The scan over a tile's groups, from the tile's first row on (BACK: from its last).
// What a lane keeps of it between its halves: the step of the parts before its own,
// and the tile's.
struct Scan {
  float A, H, tileA, tileH;
};
template <typename G, Share AS, bool BACK, bool CLEAN>
__device__ __forceinline__ Scan scan_up(const float2 *steps) {
  constexpr int N = G::N, P = G::PARTS, W = G::ACROSS;
  constexpr uint32_t FULL = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, part = lane / W, ch = lane % W;
  float2 v[N];
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = steps[G::at(part * N + j, ch)];
  Joint<AS, CLEAN> own(v[BACK ? N - 1 : 0].x, v[BACK ? N - 1 : 0].y);
#pragma unroll
  for (int k = 1; k < N; ++k) {
    const int j = BACK ? N - 1 - k : k;
    own.then(v[j].x, v[j].y);
  }
  float share = own.v(), H = own.H;
  const int behind = BACK ? P - 1 - part : part;  // parts that come before this one
#pragma unroll
  for (int o = 1; o < P; o *= 2) {
    const float v1 = BACK ? __shfl_down_sync(FULL, share, o * W) : __shfl_up_sync(FULL, share, o * W);
    const float H1 = BACK ? __shfl_down_sync(FULL, H, o * W) : __shfl_up_sync(FULL, H, o * W);
    if (behind >= o) {
      Joint<AS, CLEAN> two(v1, H1);
      two.then(share, H);
      share = two.v();
      H = two.H;
    }
  }
  const int whole = (BACK ? 0 : 32 - W) + lane % W;  // the lane that has the tile's step
  Scan s;
  s.tileA = stays<AS>(__shfl_sync(FULL, share, whole));
  s.tileH = __shfl_sync(FULL, H, whole);
  s.A = stays<AS>(BACK ? __shfl_down_sync(FULL, share, W) : __shfl_up_sync(FULL, share, W));
  s.H = BACK ? __shfl_down_sync(FULL, H, W) : __shfl_up_sync(FULL, H, W);
  if (behind == 0) {
    s.A = 1.f;
    s.H = 0.f;
  }
  return s;
}
// Replaces each group's step by the value that reaches the group, from the one that
// reaches the tile.
template <typename G, Share AS, bool BACK, bool CLEAN>
__device__ __forceinline__ void scan_down(float2 *steps, const Scan &s, float h) {
  constexpr int N = G::N, W = G::ACROSS;
  const int lane = threadIdx.x & 31, part = lane / W, ch = lane % W;
  float2 v[N];  // (all read before any is written: the compiler would keep the order)
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = steps[G::at(part * N + j, ch)];
  h = apply<CLEAN>(s.A, s.H, h);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int j = BACK ? N - 1 - k : k;
    steps[G::at(part * N + j, ch)].x = h;
    h = apply<CLEAN>(stays<AS>(v[j].x), v[j].y, h);
  }
}

// The exchange of a slab's steps among the cluster's CTAs: in each round every warp
// sends its tile's step to the warps of the CTAs that have the slab, whose barrier
// counts the bytes.  It sends those of round i + 2 after all have sent round i + 1's,
// and so have read round i's: two rounds' worth of room.
constexpr int ROOM = 2;
template <typename G>
struct Exchange {
  float2 total[ROOM][G::CLUSTER][G::SLAB];  // (1, 0) for CTAs that the cluster does not have
  uint64_t bar[ROOM];
};

__device__ __forceinline__ uint32_t peer(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// mbar_try and mbar_test for what came in from other CTAs of the cluster.
__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_test_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}

// (OTHERS: what came in is from other CTAs of the cluster)
template <bool OTHERS>
__device__ __forceinline__ bool arrived(uint32_t bar, uint32_t parity, uint64_t limit) {
  // A limit below a microsecond is a build's that tests it.  A try holds the thread until what
  // it waits for has come, if that takes no longer than a few of them: such a limit would never
  // run out.
  const bool look = limit < 1000;
  uint64_t t0 = 0;
  for (;;) {
    if (OTHERS ? (look ? mbar_test_cluster(bar, parity) : mbar_try_cluster(bar, parity))
               : (look ? mbar_test(bar, parity) : mbar_try(bar, parity)))
      return true;
    const uint64_t now = global_timer();
    if (!t0) t0 = now;
    else if (now - t0 > limit) return false;
  }
}

template <typename G>
__device__ __forceinline__ void send_step(Exchange<G> &x, int n, int rank, int i, const Scan &s, bool lost) {
  if (n == 1 || lost) return;
  const int lane = threadIdx.x & 31, ch = lane % G::ACROSS, part = lane / G::ACROSS;
  const uint32_t bar = smem_u32(&x.bar[i % ROOM]), mine = smem_u32(&x.total[i % ROOM][rank][ch]);
  if (lane == 0) mbar_expect_tx(bar, (uint32_t)n * G::SLAB * sizeof(float2));
  for (int r = part; r < n; r += G::PARTS)
    asm volatile(
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
            peer(mine, r)),
        "f"(s.tileA), "f"(s.tileH), "r"(peer(bar, r))
        : "memory");
}

// What reaches this warp's tile of round i, from the cluster's tiles' steps in the
// order of the rows (BACK: against it); `carry` is what reaches the cluster's first
// one, and then the first one of its next round.
template <typename G, bool BACK>
__device__ __forceinline__ float receive_steps(Exchange<G> &x, int n, int rank, int i, const Scan &s,
                                               float &carry, bool &lost, int32_t *status) {
  if (n == 1) {
    const float in = carry;
    carry = apply(s.tileA, s.tileH, carry);
    return in;
  }
  if (!lost) {
    const uint32_t bar = smem_u32(&x.bar[i % ROOM]), parity = (uint32_t)i / ROOM & 1;
    if (!arrived<true>(bar, parity, WAIT_LIMIT_NS)) {
      set_status(status, TWELL_ERR_TIMEOUT);
      // (what is on its way has to come in before the barrier is used again)
      lost = !arrived<true>(bar, parity, DRAIN_LIMIT_NS);
    }
    lost = __any_sync(0xFFFFFFFFu, lost);
  }
  const int ch = (threadIdx.x & 31) % G::ACROSS;
  float in = carry;
#pragma unroll
  for (int k = 0; k < G::CLUSTER; ++k) {
    const int r = BACK ? G::CLUSTER - 1 - k : k;
    if (r / 4 * 4 >= n) continue;
    if (r == rank) in = carry;
    const float2 v = x.total[i % ROOM][r][ch];
    carry = apply(v.x, v.y, carry);
  }
  return in;
}

// Before the first exchange, by the whole cluster.
template <typename G>
__device__ __forceinline__ void open_exchange(Exchange<G> &x, int C) {
  const int lane = threadIdx.x & 31;
  for (int k = lane; k < ROOM * G::CLUSTER * G::SLAB; k += 32) (&x.total[0][0][0])[k] = make_float2(1.f, 0.f);
  if (lane < ROOM) mbar_init(smem_u32(&x.bar[lane]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  if (C > 1) cluster_arrive();  // (from here on the others may write here)
}

// Rounds of a cluster's tiles.
struct Rounds {
  int C, rank, R, n;
  __device__ __forceinline__ Rounds(int C_, int rank_, int R_, int T)
      : C(C_), rank(rank_), R(R_), n(((T + R_ - 1) / R_ + C_ - 1) / C_) {}
  // first row of this CTA's tile in the i-th of them (T where it has none)
  // (T <= 2^30 and C R <= 4096: below T + C R, which fits)
  __device__ __forceinline__ int row(int i, int T) const { return min(T, (i * C + rank) * R); }
};

// What can be in a warp's tile: no sequence begins or ends there and all of its rows are
// some sequence's (PLAIN); one at most begins and one ends in each lane's rows (EASY); anything;
// no row of a sequence (DEAD).  Branches at the rows keep the rows' arithmetic from overlapping
// (in an earlier form 16384 x 2048 of 9 sequences forward 55 us, of 257 80), so what is easy has
// a selection a row instead (50 and 72).  With a gate below OPEN, which shows when the gates are read, a tile
// begins again as CLOSED: two or three selections a value, and branches at the rows.  This is a
// loop over the rows, with their gates in local memory: as much code unrolled slows the others
// down, whose own has to come from L2 when forward and backward alternate (us, loop | unrolled:
// 64 x 128 fp32 10 | 12, 4096 x 2048 of 9 sequences 49 | 63, 16384 x 4096 233 | 245).  Closed gates
// in every tile take twice a tile's time (16384 x 4096 156 + 320 | 168 + 290).  Where there is an
// EASY body, ANY goes by that loop too (sequences of 8 rows, 16384 x 2048 forward 191 us, else
// 177).
enum Kind { PLAIN_TILE, EASY_TILE, ANY_TILE, CLOSED_TILE, DEAD_TILE };
template <typename G>
__device__ __forceinline__ int kind_of(const RowBits &b) {
  if (!__any_sync(0xFFFFFFFFu, b.live != 0)) return DEAD_TILE;
  const uint32_t more = (b.first & (b.first - 1)) | (b.last & (b.last - 1));
  const bool marked = (b.first | b.last) != 0 || b.live != G::ALL;
  return __reduce_max_sync(0xFFFFFFFFu, more != 0 ? ANY_TILE : marked ? EASY_TILE : PLAIN_TILE);
}
// The last row of those marked (-1: none).
__device__ __forceinline__ int last_row(uint32_t bits) { return 31 - __clz(bits); }
// b where `other`, else a.
template <int M>
__device__ __forceinline__ void select(float2 (&a)[M], const float2 (&b)[M], bool other) {
#pragma unroll
  for (int n = 0; n < M; ++n) a[n] = make_float2(other ? b[n].x : a[n].x, other ? b[n].y : a[n].y);
}

// A tile between its two halves.
struct Tile {
  int r0;
  RowBits bits;
  int kind;
  Scan scan;
};

// What a warp of the forward has in shared memory.
template <typename G>
struct FwdShared {
  float2 steps[G::GROUPS * G::SLAB];  // the groups' steps, then what reaches them
  Exchange<G> exchange;
  // h0 of the last sequence that begins in each lane's rows: hT may be h0, and who
  // comes to that sequence's end first is open (the others end with the same lane)
  float4 held[G::N / 4][32];
  Marks<G> marks;
};

// And a CTA: x of a tile and of the next one, gates of one.
template <typename G>
struct FwdCta {
  Slot<G> x[2], gate;
  FwdShared<G> warps[WARPS];
  int32_t starts[FEW];
  uint64_t bar[2];  // of the copies of the tiles, by the tile's parity
};

// A warp of the forward.
template <typename E, int SLAB, int CLUSTER>
struct ForwardWarp {
  using G = Fwd<E, SLAB, CLUSTER>;
  static constexpr int M = G::N / 2, S = G::S, CX = G::CX;  // M pairs of channels a lane
  const E *x, *gate;
  E *h;
  const Maps &maps;
  const RecurParams &p;
  FwdCta<G> &cta;
  FwdShared<G> &sh;
  Rounds rounds;
  int C, rank, lane, q, cx, chunk, d0, d, count, lo, hi;  // d0: the CTA's first channel
  bool on, lost;
  float2 bias[M];  // times log2(e)
  float carry;  // the state before the cluster's next rows, of the scan's channel
  Gap gap;

  __device__ __forceinline__ uint32_t live_of(int i) const {
    return live_rows<S>(rounds.row(i, p.T) + q * S, lo, hi);
  }
  __device__ __forceinline__ void fetch_tile(int i) {
    if (i >= count || threadIdx.x != 0) return;
    const int r0 = rounds.row(i, p.T);
    const bool any = r0 / S < p.T / S;
    const uint32_t bar = smem_u32(&cta.bar[i & 1]);
    mbar_expect_tx(bar, any ? 2 * (uint32_t)sizeof(Slot<G>) : 0);
    if (!any) return;
    fetch(cta.x[i & 1], maps.x, r0, d0, bar);
    fetch(cta.gate, maps.gate, r0, d0, bar);
  }
  __device__ __forceinline__ void wait_tile(int i) {
    const uint32_t bar = smem_u32(&cta.bar[i & 1]), parity = (uint32_t)i >> 1 & 1;
    if (!arrived<false>(bar, parity, WAIT_LIMIT_NS)) {
      set_status(p.status, TWELL_ERR_TIMEOUT);
      arrived<false>(bar, parity, DRAIN_LIMIT_NS);  // (what is on its way has to come in)
    }
    const int r0 = rounds.row(i, p.T);
    if (p.T % S == 0 || r0 >= p.T || r0 + G::R < p.T) return;
    const int own = d - cx * G::N;
    fetch_rest(cta.x[i & 1], x, p.ld, r0, p.T, own, p.D);
    fetch_rest(cta.gate, gate, p.ld, r0, p.T, own, p.D);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  }
  __device__ __forceinline__ int slot(int k) const { return Slot<G>::at(q, k, chunk); }
  __device__ __forceinline__ void hold(const float2 (&v)[M]) {
#pragma unroll
    for (int n = 0; n < M; n += 2) sh.held[n / 2][lane] = make_float4(v[n].x, v[n].y, v[n + 1].x, v[n + 1].y);
  }
  __device__ __forceinline__ void held(float2 (&v)[M]) const {
#pragma unroll
    for (int n = 0; n < M; n += 2) {
      const float4 r = sh.held[n / 2][lane];
      v[n] = make_float2(r.x, r.y);
      v[n + 1] = make_float2(r.z, r.w);
    }
  }
  // The first half of tile i: its rows as one step a lane, scanned and sent.
  // Returns false, with nothing sent, where it finds a closed gate.
  template <int KIND>
  __device__ __forceinline__ bool first_half(int i, Tile &t, float2 (&m)[S][M]) {
    constexpr bool CLOSED = KIND == CLOSED_TILE;
    uint4 lowest;
    float2 As[M], ns[M], Hs[M];  // the rows so far, see Joint
#pragma unroll
    for (int n = 0; n < M; ++n) {
      As[n] = both(1.f);
      ns[n] = both(NOTHING);
      Hs[n] = both(0.f);
    }
    float2 start[M] = {};
    const int begin = KIND == EASY_TILE ? last_row(t.bits.first) : -1;
    if (KIND == EASY_TILE && begin >= 0) {
      load_state(on ? p.h0 : nullptr, first_of(p, sh.marks, t.r0, q * S + begin), p.D, d, start);
      hold(start);
    }
#pragma unroll(CLOSED ? 1 : S)
    for (int k = 0; k < S; ++k) {
      if (KIND == EASY_TILE) select(Hs, start, k == begin);
      if (KIND >= ANY_TILE && (t.bits.any_first >> k & 1) && (t.bits.first >> k & 1)) {
        load_state(on ? p.h0 : nullptr, first_of(p, sh.marks, t.r0, q * S + k), p.D, d, Hs);
        hold(Hs);
      }
      float2 xv[M], gv[M];
      pairs(cta.x[i & 1].v[slot(k)], xv, (E *)nullptr);
      const uint4 gates = cta.gate.v[slot(k)];
      if (!CLOSED) lowest = k == 0 ? gates : lower(lowest, gates, (E *)nullptr);
      pairs(gates, gv, (E *)nullptr);
#pragma unroll
      for (int n = 0; n < M; ++n) {
        const float2 g = fma2(gv[n], both(LOG2E), bias[n]);
        m[k][n] = gate_of<CLOSED>(g, exp2_of(g));
        Hs[n] = row_step<CLOSED>(m[k][n], xv[n], Hs[n], less2(Hs[n], xv[n]));
        ns[n] = fma2(m[k][n], As[n], ns[n]);
        As[n] = kept<CLOSED>(m[k][n], As[n]);
      }
    }
    if (!CLOSED) {
      float2 gv[M];
      pairs(lowest, gv, (E *)nullptr);
      bool closed = false;
#pragma unroll
      for (int n = 0; n < M; ++n) {
        const float2 t = fma2(gv[n], both(LOG2E), bias[n]);
        closed |= fminf(t.x, t.y) < OPEN;
      }
      if (__any_sync(0xFFFFFFFFu, closed)) return false;
    }
    cta_barrier();  // (all warps are done with the gates, and with tile i - 1)
    fetch_tile(i + 1);
    const bool cut = KIND != PLAIN_TILE && (t.bits.first != 0 || t.bits.live != G::ALL);
#pragma unroll
    for (int n = 0; n < M; ++n) {
      const float2 all = make_float2(smaller(As[n].x, ns[n].x), smaller(As[n].y, ns[n].y));
      sh.steps[G::at(q, 2 * n * CX + cx)] = make_float2(cut ? CUT : all.x, Hs[n].x);
      sh.steps[G::at(q, (2 * n + 1) * CX + cx)] = make_float2(cut ? CUT : all.y, Hs[n].y);
    }
    __syncwarp();
    t.scan = scan_up<G, AS_M, false, KIND == PLAIN_TILE>(sh.steps);
    send_step<G>(sh.exchange, C, rank, i, t.scan, lost);
    return true;
  }
  // A tile without a row of any sequence.
  __device__ __forceinline__ void skip(int i, Tile &t) {
    cta_barrier();
    fetch_tile(i + 1);
    t.scan.tileA = CUT;
    t.scan.tileH = 0.f;
    send_step<G>(sh.exchange, C, rank, i, t.scan, lost);
    receive_steps<G, false>(sh.exchange, C, rank, i, t.scan, carry, lost, p.status);
  }
  // The second half: the rows once more, from the state before them.
  template <int KIND>
  __device__ __forceinline__ void second_half(int i, const Tile &t, const float2 (&m)[S][M]) {
    constexpr bool CLOSED = KIND == CLOSED_TILE;
    const float in = receive_steps<G, false>(sh.exchange, C, rank, i, t.scan, carry, lost, p.status);
    scan_down<G, AS_M, false, KIND == PLAIN_TILE>(sh.steps, t.scan, in);
    __syncwarp();
    float2 y[M];
#pragma unroll
    for (int n = 0; n < M; ++n)
      y[n] = make_float2(sh.steps[G::at(q, 2 * n * CX + cx)].x,
                         sh.steps[G::at(q, (2 * n + 1) * CX + cx)].x);
    if (!on) return;
    const int row = t.r0 + q * S;
    if (p.states && row % RECUR_KEEP == 0 && row < p.T)
      store_state(p.states, row / RECUR_KEEP, p.D, d, y);
    E *out = h + (size_t)row * p.D + d;
    float2 start[M] = {}, behind[M] = {};
    const int begin = KIND == EASY_TILE ? last_row(t.bits.first) : -1;
    const int end = KIND == EASY_TILE ? last_row(t.bits.last) : -1;
    if (KIND == EASY_TILE) held(start);
    uint4 rows[CLOSED ? 1 : S];  // (read before the first store, which the reads could not pass)
#pragma unroll
    for (int k = 0; !CLOSED && k < S; ++k) rows[CLOSED ? 0 : k] = cta.x[i & 1].v[slot(k)];
#pragma unroll(CLOSED ? 1 : S)
    for (int k = 0; k < S; ++k, out += p.D) {
      float2 xv[M];
      pairs(CLOSED ? cta.x[i & 1].v[slot(k)] : rows[CLOSED ? 0 : k], xv, (E *)nullptr);
      if (KIND == EASY_TILE) select(y, start, k == begin);
      if (KIND >= ANY_TILE && (t.bits.any_first >> k & 1)) {
        if (t.bits.first >> k == 1) held(y);
        else if (t.bits.first >> k & 1) load_state(p.h0, first_of(p, sh.marks, t.r0, q * S + k), p.D, d, y);
      }
#pragma unroll
      for (int n = 0; n < M; ++n) y[n] = row_step<CLOSED>(m[k][n], xv[n], y[n], less2(y[n], xv[n]));
      if (KIND == PLAIN_TILE || (t.bits.live >> k & 1)) *(uint4 *)out = packed(y, (E *)nullptr);
      if (KIND == EASY_TILE) select(behind, y, k == end);
      if (KIND >= ANY_TILE && (t.bits.any_last >> k & 1) && (t.bits.last >> k & 1) && p.hT)
        store_state(p.hT, last_of(p, sh.marks, t.r0, q * S + k), p.D, d, y);
    }
    if (KIND == EASY_TILE && end >= 0 && p.hT)
      store_state(p.hT, last_of(p, sh.marks, t.r0, q * S + end), p.D, d, behind);
  }
};

template <typename E, int SLAB, int CLUSTER>
__global__ void __launch_bounds__(32 * WARPS, CLUSTER == 8 || sizeof(E) == 4 ? 3 : 2)
recur_forward_kernel(const E *x, const E *gate, E *h, const __grid_constant__ Maps maps, RecurParams p) {
  pdl_begin();
  using G = Fwd<E, SLAB, CLUSTER>;
  extern __shared__ __align__(1024) char shared[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  FwdCta<G> &cta = *(FwdCta<G> *)shared;
  FwdShared<G> &sh = cta.warps[warp];
  const int32_t *starts = keep_starts(p, cta.starts);
  open_exchange(sh.exchange, C);
  const int base = (int)(blockIdx.x / C) * WARPS * G::SLAB, d0 = base + warp * G::SLAB;
  const Rounds rounds(C, rank, G::R, p.T);
  const int q = Slot<G>::group(lane / G::CX), cx = lane % G::CX, d = d0 + cx * G::N, count = rounds.n;
  const int lo = p.starts ? max(0, p.starts[0]) : 0;
  const int hi = p.starts ? min(p.T, max(0, p.starts[p.B])) : p.T;
  ForwardWarp<E, SLAB, CLUSTER> w{x, gate, h, maps, p, cta, sh, rounds, C, rank, lane, q, cx, warp * G::CX + cx, base, d, count, lo, hi, d < p.D, false};
  if (threadIdx.x < 2) mbar_init(smem_u32(&cta.bar[threadIdx.x]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  cta_barrier();
  w.fetch_tile(0);
  empty_sequences(p, p.h0, p.hT, d0, min(p.D, d0 + G::SLAB), rank, C);
  load_state(w.on ? p.bias : nullptr, 0, 0, d, w.bias);
#pragma unroll
  for (int n = 0; n < G::N / 2; ++n) w.bias[n] = mul2(w.bias[n], both(LOG2E));
  w.carry = 0.f;
  if (C > 1) cluster_wait();
  Tile t;
  float2 c[G::S][G::N / 2];
  for (int i = 0; i < count; ++i) {
    t.r0 = rounds.row(i, p.T);
    t.kind = PLAIN_TILE;
    t.bits = RowBits{0, 0, G::ALL, 0, 0};
    if (!plain_tile<G::R>(p, w.gap, t.r0, lo, hi)) {
      t.bits = row_bits(p, starts, sh.marks, w.gap, t.r0, q, w.live_of(i));
      t.kind = kind_of<G>(t.bits);
    }
    w.wait_tile(i);
    if (t.kind == PLAIN_TILE && w.template first_half<PLAIN_TILE>(i, t, c)) {
      w.template second_half<PLAIN_TILE>(i, t, c);
    } else if (t.kind == EASY_TILE && w.template first_half<EASY_TILE>(i, t, c)) {
      w.template second_half<EASY_TILE>(i, t, c);
    } else if (t.kind == DEAD_TILE) {
      w.skip(i, t);
    } else {
      float2 cc[G::S][G::N / 2];
      w.template first_half<CLOSED_TILE>(i, t, cc);
      w.template second_half<CLOSED_TILE>(i, t, cc);
    }
  }
  // (nothing is on its way to this CTA any more, unless a wait has given up)
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  }
}

// What a warp of the backward has in shared memory.
template <typename G>
struct BwdShared {
  float2 stepsF[G::GROUPS * G::SLAB];     // the groups' steps forward
  float2 stepsB[G::GROUPS * G::SLAB];  // and back, then what reaches them
  Exchange<G> exchange;
  float bias[G::CLUSTER][G::SLAB];       // the CTAs' sums of dgate
  Marks<G> marks;
};

template <typename G>
struct BwdCta {
  // x of a tile and of the next one, where that costs no CTA of the SM (16384 x 4096: 150
  // us, else 156; 16384 x 2048 of 65 sequences, with two CTAs where there were three: 142, else
  // 124)
  static constexpr int XS = G::SLAB == 16 && G::CLUSTER == 16 ? 1 : 2;
  Slot<G> x[XS], gate, dh[2];
  BwdShared<G> warps[WARPS];
  int32_t starts[FEW];
  uint64_t bar[2];  // of the copies of the tiles, by the tile's parity
};

// A warp of the backward, which goes from the last tile to the first.
template <typename E, int SLAB, int S, int CLUSTER>
struct BackwardWarp {
  using G = Bwd<E, SLAB, S, CLUSTER>;
  static constexpr int M = G::N / 2, CX = G::CX, XS = BwdCta<G>::XS;
  const E *x, *gate, *dh;
  E *dx, *dgate;
  const Maps &maps;
  const RecurParams &p;
  BwdCta<G> &cta;
  BwdShared<G> &sh;
  Rounds rounds;
  int C, rank, lane, q, cx, chunk, d0, d, sd, count, lo, hi;  // d0: the CTA's first channel, sd: the scan's
  bool on, lost;
  float2 bias[M], db[M];
  float carry;   // a G behind the cluster's next rows, of the scan's channel
  float before;  // the state before the next tile
  Gap gap;

  __device__ __forceinline__ int first_row(int i) const { return rounds.row(rounds.n - 1 - i, p.T); }
  __device__ __forceinline__ uint32_t live_of(int i) const {
    return live_rows<S>(first_row(i) + q * S, lo, hi);
  }
  // A tile's copies; x's apart where its only slot is free later than the gates'.
  __device__ __forceinline__ void fetch_tile(int i) {
    if (i >= count || threadIdx.x != 0) return;
    const int r0 = first_row(i);
    const bool any = r0 / S < p.T / S;
    const uint32_t bar = smem_u32(&cta.bar[i & 1]);
    mbar_expect_tx(bar, any ? 3 * (uint32_t)sizeof(Slot<G>) : 0);
    if (!any) return;
    fetch(cta.gate, maps.gate, r0, d0, bar);
    fetch(cta.dh[i & 1], maps.dh, r0, d0, bar);
    if (XS == 2) fetch(cta.x[i % XS], maps.x, r0, d0, bar);
  }
  __device__ __forceinline__ void fetch_x(int i) {
    if (i >= count || threadIdx.x != 0) return;
    const int r0 = first_row(i);
    if (r0 / S < p.T / S) fetch(cta.x[i % XS], maps.x, r0, d0, smem_u32(&cta.bar[i & 1]));
  }
  __device__ __forceinline__ void wait_tile(int i) {
    const uint32_t bar = smem_u32(&cta.bar[i & 1]), parity = (uint32_t)i >> 1 & 1;
    if (!arrived<false>(bar, parity, WAIT_LIMIT_NS)) {
      set_status(p.status, TWELL_ERR_TIMEOUT);
      arrived<false>(bar, parity, DRAIN_LIMIT_NS);  // (what is on its way has to come in)
    }
    const int r0 = first_row(i);
    if (p.T % S == 0 || r0 >= p.T || r0 + G::R < p.T) return;
    const int own = d - cx * G::N;
    fetch_rest(cta.x[i % XS], x, p.ld, r0, p.T, own, p.D);
    fetch_rest(cta.gate, gate, p.ld, r0, p.T, own, p.D);
    fetch_rest(cta.dh[i & 1], dh, (long long)p.D, r0, p.T, own, p.D);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  }
  __device__ __forceinline__ int slot(int k) const { return Slot<G>::at(q, k, chunk); }
  // (where a tile's first row begins a sequence it is not used)
  __device__ __forceinline__ float state_before(int i) const {
    const int r0 = i < count ? first_row(i) : p.T;
    return sd < p.D && r0 > 0 && r0 < p.T ? p.states[(size_t)(r0 / RECUR_KEEP) * p.D + sd] : 0.f;
  }
  // The first half of tile i: its rows as one step forward and one back; h within the
  // tile needs no other, and of the gates there stay m and e := (h_{t-1} - x_t) a c.
  template <int KIND>
  __device__ __forceinline__ bool first_half(int i, Tile &t, float2 (&e)[S][M], float2 (&m)[S][M]) {
    constexpr bool CLOSED = KIND == CLOSED_TILE;
    uint4 lowest;
    float2 As[M], ns[M], Hs[M];  // the rows so far, see Joint
#pragma unroll
    for (int n = 0; n < M; ++n) {
      As[n] = both(1.f);
      ns[n] = both(NOTHING);
      Hs[n] = both(0.f);
    }
    float2 start[M] = {};
    const int begin = KIND == EASY_TILE ? last_row(t.bits.first) : -1;
    const int end = KIND == EASY_TILE ? last_row(t.bits.last) : -1;
    const auto at_begin = [&](float2 (&v)[M]) {
      if (KIND == EASY_TILE && begin >= 0)
        load_state(on ? p.h0 : nullptr, first_of(p, sh.marks, t.r0, q * S + begin), p.D, d, v);
    };
    at_begin(start);
#pragma unroll(CLOSED ? 1 : S)
    for (int k = 0; k < S; ++k) {
      if (KIND == EASY_TILE) select(Hs, start, k == begin);
      if (KIND >= ANY_TILE && (t.bits.any_first >> k & 1) && (t.bits.first >> k & 1))
        load_state(on ? p.h0 : nullptr, first_of(p, sh.marks, t.r0, q * S + k), p.D, d, Hs);
      float2 xv[M], gv[M];
      pairs(cta.x[i % XS].v[slot(k)], xv, (E *)nullptr);
      const uint4 gates = cta.gate.v[slot(k)];
      if (!CLOSED) lowest = k == 0 ? gates : lower(lowest, gates, (E *)nullptr);
      pairs(gates, gv, (E *)nullptr);
#pragma unroll
      for (int n = 0; n < M; ++n) {
        const float2 g = fma2(gv[n], both(LOG2E), bias[n]), eg = exp2_held(g);
        m[k][n] = gate_of<CLOSED>(g, eg);
        e[k][n] = both_shares<CLOSED>(g, eg, m[k][n]);
        Hs[n] = row_step<CLOSED>(m[k][n], xv[n], Hs[n], less2(Hs[n], xv[n]));
        ns[n] = fma2(m[k][n], As[n], ns[n]);
        As[n] = kept<CLOSED>(m[k][n], As[n]);
      }
    }
    if (!CLOSED) {
      float2 gv[M];
      pairs(lowest, gv, (E *)nullptr);
      bool closed = false;
#pragma unroll
      for (int n = 0; n < M; ++n) {
        const float2 t = fma2(gv[n], both(LOG2E), bias[n]);
        closed |= fminf(t.x, t.y) < OPEN;
      }
      if (__any_sync(0xFFFFFFFFu, closed)) return false;
    }
    cta_barrier();  // (all warps are done with the gates, and with the last tile's dh)
    fetch_tile(i + 1);
    const bool dead = KIND != PLAIN_TILE && t.bits.live != G::ALL;
    const bool cutF = KIND != PLAIN_TILE && (dead || t.bits.first),
               cutB = KIND != PLAIN_TILE && (dead || t.bits.last);
#pragma unroll
    for (int n = 0; n < M; ++n) {
      sh.stepsF[G::at(q, 2 * n * CX + cx)] = make_float2(cutF ? CUT : As[n].x, Hs[n].x);
      sh.stepsF[G::at(q, (2 * n + 1) * CX + cx)] = make_float2(cutF ? CUT : As[n].y, Hs[n].y);
      As[n] = make_float2(smaller(As[n].x, ns[n].x), smaller(As[n].y, ns[n].y));
      Hs[n] = both(0.f);
    }
    if (KIND == EASY_TILE && end >= 0)
      load_state(on ? p.dhT : nullptr, last_of(p, sh.marks, t.r0, q * S + end), p.D, d, start);
#pragma unroll(CLOSED ? 1 : S)
    for (int k = S - 1; k >= 0; --k) {
      if (KIND == EASY_TILE) select(Hs, start, k == end);
      if (KIND >= ANY_TILE && (t.bits.any_last >> k & 1) && (t.bits.last >> k & 1))
        load_state(on ? p.dhT : nullptr, last_of(p, sh.marks, t.r0, q * S + k), p.D, d, Hs);
      float2 dv[M];
      pairs(cta.dh[i & 1].v[slot(k)], dv, (E *)nullptr);
#pragma unroll
      for (int n = 0; n < M; ++n) {
        Hs[n] = kept<CLOSED>(m[k][n], add2(dv[n], Hs[n]));
      }
    }
#pragma unroll
    for (int n = 0; n < M; ++n) {
      sh.stepsB[G::at(q, 2 * n * CX + cx)] = make_float2(cutB ? CUT : As[n].x, Hs[n].x);
      sh.stepsB[G::at(q, (2 * n + 1) * CX + cx)] = make_float2(cutB ? CUT : As[n].y, Hs[n].y);
    }
    __syncwarp();
    t.scan = scan_up<G, AS_M, true, KIND == PLAIN_TILE>(sh.stepsB);
    send_step<G>(sh.exchange, C, rank, i, t.scan, lost);
    scan_down<G, AS_A, false, KIND == PLAIN_TILE>(
        sh.stepsF, scan_up<G, AS_A, false, KIND == PLAIN_TILE>(sh.stepsF), before);
    before = state_before(i + 1);
    __syncwarp();
    float2 y[M];
#pragma unroll
    for (int n = 0; n < M; ++n)
      y[n] = make_float2(sh.stepsF[G::at(q, 2 * n * CX + cx)].x, sh.stepsF[G::at(q, (2 * n + 1) * CX + cx)].x);
    at_begin(start);
#pragma unroll(CLOSED ? 1 : S)
    for (int k = 0; k < S; ++k) {
      if (KIND == EASY_TILE) select(y, start, k == begin);
      if (KIND >= ANY_TILE && (t.bits.any_first >> k & 1) && on && (t.bits.first >> k & 1))
        load_state(p.h0, first_of(p, sh.marks, t.r0, q * S + k), p.D, d, y);
      float2 xv[M];
      pairs(cta.x[i % XS].v[slot(k)], xv, (E *)nullptr);
#pragma unroll
      for (int n = 0; n < M; ++n) {
        const float2 off = less2(y[n], xv[n]);
        y[n] = row_step<CLOSED>(m[k][n], xv[n], y[n], off);
        e[k][n] = mul2(off, e[k][n]);
      }
    }
    if constexpr (XS == 1) {
      cta_barrier();  // (all warps are done with x)
      fetch_x(i + 1);
    }
    return true;
  }
  // A tile without a row of any sequence.
  __device__ __forceinline__ void skip(int i, Tile &t) {
    cta_barrier();
    fetch_tile(i + 1);
    if (XS == 1) fetch_x(i + 1);  // (which no warp reads here)
    before = state_before(i + 1);
    t.scan.tileA = CUT;
    t.scan.tileH = 0.f;
    send_step<G>(sh.exchange, C, rank, i, t.scan, lost);
    receive_steps<G, true>(sh.exchange, C, rank, i, t.scan, carry, lost, p.status);
  }
  // The second half: G, from the last row on.
  template <int KIND>
  __device__ __forceinline__ void second_half(int i, const Tile &t, const float2 (&e)[S][M],
                                              const float2 (&m)[S][M]) {
    constexpr bool CLOSED = KIND == CLOSED_TILE;
    const float in = receive_steps<G, true>(sh.exchange, C, rank, i, t.scan, carry, lost, p.status);
    scan_down<G, AS_M, true, KIND == PLAIN_TILE>(sh.stepsB, t.scan, in);
    __syncwarp();
    float2 y[M];
#pragma unroll
    for (int n = 0; n < M; ++n)
      y[n] = make_float2(sh.stepsB[G::at(q, 2 * n * CX + cx)].x,
                         sh.stepsB[G::at(q, (2 * n + 1) * CX + cx)].x);
    if (!on) return;
    const int row = t.r0 + q * S;
    E *px = dx + (size_t)row * p.ld + d, *pg = dgate + (size_t)row * p.ld + d;
    uint4 rows[CLOSED ? 1 : S];
#pragma unroll
    for (int k = 0; !CLOSED && k < S; ++k) rows[CLOSED ? 0 : k] = cta.dh[i & 1].v[slot(k)];
    float2 start[M] = {}, ahead[M] = {};
    const int begin = KIND == EASY_TILE ? last_row(t.bits.first) : -1;
    const int end = KIND == EASY_TILE ? last_row(t.bits.last) : -1;
    if (KIND == EASY_TILE && end >= 0)
      load_state(p.dhT, last_of(p, sh.marks, t.r0, q * S + end), p.D, d, start);
#pragma unroll(CLOSED ? 1 : S)
    for (int k = S - 1; k >= 0; --k) {
      if (KIND == EASY_TILE) select(y, start, k == end);
      if (KIND >= ANY_TILE && (t.bits.any_last >> k & 1) && (t.bits.last >> k & 1))
        load_state(p.dhT, last_of(p, sh.marks, t.r0, q * S + k), p.D, d, y);
      const bool live = KIND == PLAIN_TILE || (t.bits.live >> k & 1);
      float2 dv[M], gv[M];
      pairs(CLOSED ? cta.dh[i & 1].v[slot(k)] : rows[CLOSED ? 0 : k], dv, (E *)nullptr);
#pragma unroll
      for (int n = 0; n < M; ++n) {
        const float2 g = add2(dv[n], y[n]);
        gv[n] = mul2(g, e[k][n]);
        if (live) db[n] = add2(db[n], gv[n]);
        dv[n] = minus_taken<CLOSED>(m[k][n], g);
        y[n] = kept<CLOSED>(m[k][n], g);
      }
      if (live) {
        *(uint4 *)(px + k * p.ld) = packed<true>(dv, (E *)nullptr);
        *(uint4 *)(pg + k * p.ld) = packed(gv, (E *)nullptr);
      }
      if (KIND == EASY_TILE) select(ahead, y, k == begin);
      if (KIND >= ANY_TILE && (t.bits.any_first >> k & 1) && (t.bits.first >> k & 1) && p.dh0)
        store_state(p.dh0, first_of(p, sh.marks, t.r0, q * S + k), p.D, d, y);
    }
    if (KIND == EASY_TILE && begin >= 0 && p.dh0)
      store_state(p.dh0, first_of(p, sh.marks, t.r0, q * S + begin), p.D, d, ahead);
  }
};

template <typename E, int SLAB, int S, int CLUSTER>
__global__ void __launch_bounds__(32 * WARPS, S == 4 ? 3 : 2)
recur_backward_kernel(const E *x, const E *gate, const E *dh, E *dx, E *dgate, const __grid_constant__ Maps maps, RecurParams p) {
  pdl_begin();
  using G = Bwd<E, SLAB, S, CLUSTER>;
  constexpr int N = G::N, CX = G::CX;
  extern __shared__ __align__(1024) char shared[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  BwdCta<G> &cta = *(BwdCta<G> *)shared;
  BwdShared<G> &sh = cta.warps[warp];
  const int32_t *starts = keep_starts(p, cta.starts);
  open_exchange(sh.exchange, C);
  const int base = (int)(blockIdx.x / C) * WARPS * G::SLAB, d0 = base + warp * G::SLAB;
  const Rounds rounds(C, rank, G::R, p.T);
  const int q = Slot<G>::group(lane / CX), cx = lane % CX, d = d0 + cx * N, count = rounds.n;
  const int sc = lane % G::ACROSS, sd = d0 + sc % CX * N + sc / CX;
  const int lo = p.starts ? max(0, p.starts[0]) : 0;
  const int hi = p.starts ? min(p.T, max(0, p.starts[p.B])) : p.T;
  BackwardWarp<E, SLAB, S, CLUSTER> w{x, gate, dh, dx, dgate, maps, p, cta, sh, rounds, C, rank, lane, q, cx, warp * CX + cx, base, d, sd, count, lo, hi, d < p.D, false};
  if (threadIdx.x < 2) mbar_init(smem_u32(&cta.bar[threadIdx.x]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  cta_barrier();
  w.fetch_tile(0);
  if (BwdCta<G>::XS == 1) w.fetch_x(0);
  w.before = w.state_before(0);
  empty_sequences(p, p.dhT, p.dh0, d0, min(p.D, d0 + G::SLAB), rank, C);
  load_state(w.on ? p.bias : nullptr, 0, 0, d, w.bias);
#pragma unroll
  for (int n = 0; n < N / 2; ++n) {
    w.bias[n] = mul2(w.bias[n], both(LOG2E));
    w.db[n] = both(0.f);
  }
  w.carry = 0.f;
  if (C > 1) cluster_wait();
  // (with 8 rows of bf16 an easy body costs all of them registers: 16384 x 512 43 us, with it
  // 46)
  constexpr bool EASY = sizeof(E) == 4 || S == 4;
  constexpr int MARKED = EASY ? EASY_TILE : ANY_TILE;
  Tile t;
  float2 c[G::S][N / 2], e[G::S][N / 2];
  for (int i = 0; i < count; ++i) {
    t.r0 = w.first_row(i);
    t.kind = PLAIN_TILE;
    t.bits = RowBits{0, 0, G::ALL, 0, 0};
    if (!plain_tile<G::R>(p, w.gap, t.r0, lo, hi)) {
      t.bits = row_bits(p, starts, sh.marks, w.gap, t.r0, q, w.live_of(i));
      t.kind = kind_of<G>(t.bits);
    }
    w.wait_tile(i);
    if (t.kind == PLAIN_TILE && w.template first_half<PLAIN_TILE>(i, t, e, c)) {
      w.template second_half<PLAIN_TILE>(i, t, e, c);
    } else if (t.kind == DEAD_TILE) {
      w.skip(i, t);
    } else if (t.kind != PLAIN_TILE && !(EASY && t.kind == ANY_TILE) &&
               w.template first_half<MARKED>(i, t, e, c)) {
      w.template second_half<MARKED>(i, t, e, c);
    } else {
      float2 cc[G::S][N / 2], ce[G::S][N / 2];
      w.template first_half<CLOSED_TILE>(i, t, ce, cc);
      w.template second_half<CLOSED_TILE>(i, t, ce, cc);
    }
  }
  float db[N];
#pragma unroll
  for (int n = 0; n < N; ++n) db[n] = n & 1 ? w.db[n / 2].y : w.db[n / 2].x;
  // the bias' gradient: the warp's groups, then the CTAs, in order
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int o = 16; o >= CX; o /= 2) db[n] += __shfl_down_sync(0xFFFFFFFFu, db[n], o);
    if (lane < CX) *cluster.map_shared_rank(&sh.bias[rank][cx * N + n], 0) = db[n];
  }
  cluster_arrive();
  cluster_wait();
  if (rank != 0 || !p.dbias || lane >= G::SLAB || d0 + lane >= p.D) return;
  float sum = 0.f;
  for (int r = 0; r < C; ++r) sum += sh.bias[r][lane];
  p.dbias[d0 + lane] = sum;
}

// Sequences of one row (a decoded token each): a thread for 16 bytes.
constexpr int STEP_THREADS = 128;

template <typename E>
__global__ void __launch_bounds__(STEP_THREADS)
recur_step_kernel(const E *x, const E *gate, E *h, RecurParams p) {
  pdl_begin();
  constexpr int N = VEC16<E>;
  const int per = p.D / N;
  const long long k = (long long)blockIdx.x * STEP_THREADS + threadIdx.x;
  const int row = (int)(k / per), d = (int)(k % per) * N;
  if (row >= p.T) return;
  constexpr int M = N / 2;
  float2 xv[M], gv[M], y[M], bias[M];
  pairs(*(const uint4 *)(x + (size_t)row * p.ld + d), xv, (E *)nullptr);
  pairs(*(const uint4 *)(gate + (size_t)row * p.ld + d), gv, (E *)nullptr);
  load_state(p.bias, 0, 0, d, bias);
  load_state(p.h0, row, p.D, d, y);
#pragma unroll
  for (int n = 0; n < M; ++n) {
    const float2 t = fma2(gv[n], both(LOG2E), mul2(bias[n], both(LOG2E)));
    y[n] = row_step<true>(gate_of<true>(t, exp2_of(t)), xv[n], y[n], less2(y[n], xv[n]));
  }
  *(uint4 *)(h + (size_t)row * p.D + d) = packed(y, (E *)nullptr);
  if (p.hT) store_state(p.hT, row, p.D, d, y);
}

RecurParams params_of(const RecurArgs &a) {
  RecurParams p;
  p.starts = a.starts; p.B = a.B; p.T = a.T; p.D = a.D; p.len = a.T / a.B; p.ld = a.ld;
  p.bias = a.bias; p.h0 = a.h0; p.hT = a.hT; p.states = a.states; p.dhT = a.dhT;
  p.dbias = a.dbias; p.dh0 = a.dh0; p.status = a.status;
  return p;
}

// The matrix of pitch ld at v as tensor of (channel, group, row of the group), in tiles
// of Slot<G>.
template <typename G>
bool map_of(CUtensorMap &map, const void *v, long long ld, int T, int D) {
  constexpr int CH = Slot<G>::CH;
  const EncodeFn encode = encode_fn();
  if (!encode) return false;
  constexpr cuuint64_t SIZE = 16 / G::N;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)(T < G::S ? 1 : T / G::S), (cuuint64_t)G::S};
  const cuuint64_t pitch[2] = {(cuuint64_t)ld * G::S * SIZE, (cuuint64_t)ld * SIZE};
  const cuuint32_t box[3] = {(cuuint32_t)CH * G::N, (cuuint32_t)G::GROUPS, (cuuint32_t)G::S};
  const cuuint32_t step[3] = {1, 1, 1};
  return encode(&map, SIZE == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                const_cast<void *>(v), dims, pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CH == 8 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of C CTAs of a kernel that are resident at once (0: cannot be told).
template <typename K>
int resident_clusters(K kern, int threads, size_t smem, int C) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C);
  cfg.blockDim = dim3((unsigned)threads);
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

// A kernel's clusters: as few CTAs as make the fewest rounds, while all of them are
// resident at once.
template <typename K, int MOST>
struct Shape {
  cudaError_t attr;
  int fit[MOST + 1];  // clusters that are resident, by their CTAs
  Shape(K kern, int threads, size_t smem)
      : attr(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) {
    if (attr == cudaSuccess && MOST > 8)
      attr = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (int C = 1; C <= MOST; ++C)
      fit[C] = attr == cudaSuccess ? resident_clusters(kern, threads, smem, C) : 0;
  }
  int cluster(int ctas, int tiles) const {
    int C = 1;
    for (int k = 2; k <= MOST && k <= tiles; ++k)
      if (fit[k] >= ctas && (tiles + k - 1) / k < (tiles + C - 1) / C) C = k;
    return C;
  }
};

// bf16 takes 16 channels a warp where clusters of 16 CTAs of that width fill the SMs, two
// CTAs each; else 8, which double the CTAs (us, 8 | 16: 16384 x 512 forward + backward
// 24 + 45 | 30 + 60, 131072 x 1024 forward 193 | 214, 16384 x 1280 49 + 93 | 42 + 78, 16384 x
// 4096 100 + 203 | 81 + 150: 16 bytes of a row are half a sector).  fp32 always 8 (in an earlier
// form 8192 x 4096 79 + 138 | 77 + 148, 2048 x 1024 10 + 14 | 14 + 22).
int columns(int D) { return (D + 63) / 64; }
bool wide(int D) { return columns(D) * 16 >= 2 * num_sms(); }
// Clusters of 8 leave room in shared memory for a third CTA of the forward and for more
// copies on their way in the backward, where there are the CTAs (8 | 16: 16384 x 4096 81 +
// 150 | 89 + 158, 16384 x 2048 of 9 sequences 55 + 100 | 54 + 94, 16384 x 1536 55 + 99 | 47 + 81).
bool wider(int D) { return columns(D) * 8 > 2 * num_sms(); }

template <typename E, int SLAB, int CLUSTER>
cudaError_t forward_w(const RecurArgs &a, cudaStream_t s) {
  using G = Fwd<E, SLAB, CLUSTER>;
  constexpr int SMEM = sizeof(FwdCta<G>);
  auto kern = recur_forward_kernel<E, SLAB, CLUSTER>;
  static const Shape<decltype(kern), G::CLUSTER> shape(kern, 32 * WARPS, SMEM);
  if (shape.attr != cudaSuccess) return shape.attr;
  const int width = WARPS * G::SLAB, ctas = (a.D + width - 1) / width;
  const int C = shape.cluster(ctas, (a.T + G::R - 1) / G::R);
  Maps maps;
  if (!map_of<G>(maps.x, a.x, a.ld, a.T, a.D) ||
      !map_of<G>(maps.gate, a.gate, a.ld, a.T, a.D))
    return cudaErrorNotSupported;
  maps.dh = maps.x;
  return launch_clusters(kern, dim3((unsigned)(ctas * C)), dim3(32 * WARPS), SMEM, C, s,
                         (const E *)a.x, (const E *)a.gate, (E *)a.h, maps, params_of(a));
}

template <typename E>
cudaError_t forward_t(const RecurArgs &a, cudaStream_t s) {
  if (!a.starts && a.B == a.T) {
    const long long vecs = (long long)a.T * (a.D / VEC16<E>);
    return launch_k(recur_step_kernel<E>, dim3((unsigned)((vecs + STEP_THREADS - 1) / STEP_THREADS)),
                    dim3(STEP_THREADS), 0, s, (const E *)a.x, (const E *)a.gate, (E *)a.h,
                    params_of(a));
  }
  if constexpr (sizeof(E) == 2)
    if (wide(a.D) || (a.starts && a.B > MAX_SHORT_B))
      return wider(a.D) ? forward_w<E, 16, 8>(a, s) : forward_w<E, 16, 16>(a, s);
  return forward_w<E, 8, 16>(a, s);
}

template <typename E, int SLAB, int S, int CLUSTER>
cudaError_t backward_s(const RecurArgs &a, cudaStream_t s) {
  using G = Bwd<E, SLAB, S, CLUSTER>;
  constexpr int SMEM = sizeof(BwdCta<G>);
  auto kern = recur_backward_kernel<E, SLAB, S, CLUSTER>;
  static const Shape<decltype(kern), G::CLUSTER> shape(kern, 32 * WARPS, SMEM);
  if (shape.attr != cudaSuccess) return shape.attr;
  const int width = WARPS * G::SLAB, ctas = (a.D + width - 1) / width;
  const int C = shape.cluster(ctas, (a.T + G::R - 1) / G::R);
  Maps maps;
  if (!map_of<G>(maps.x, a.x, a.ld, a.T, a.D) ||
      !map_of<G>(maps.gate, a.gate, a.ld, a.T, a.D) ||
      !map_of<G>(maps.dh, a.dh, a.D, a.T, a.D))
    return cudaErrorNotSupported;
  return launch_clusters(kern, dim3((unsigned)(ctas * C)), dim3(32 * WARPS), SMEM, C, s,
                         (const E *)a.x, (const E *)a.gate, (const E *)a.dh, (E *)a.dx, (E *)a.dgate,
                         maps, params_of(a));
}


// Tiles of 4 rows a group leave room for a third CTA; those of 8 have fewer rounds, each of a
// fixed cost.  With 16 channels a warp 4 rows win at every number of sequences; with 8 in
// calls of few rows (us, 4 | 8: 64 x 128 fp32 5.8 | 11, 16384 x 2048 of 1 sequence 84 | 85, of 9
// 93 | 106, of 65 124 | 178, 16384 x 4096 149 | 151; 8 channels, 16384 x 512 46 | 45, 16384 x 128
// of 50 36 | 34, 16384 x 512 of 65 fp32 75 | 61).
constexpr int FEW_ROWS = 4096;

template <typename E, int SLAB, int CLUSTER>
cudaError_t backward_w(const RecurArgs &a, cudaStream_t s) {
  if constexpr (SLAB == 8)
    if (a.T > FEW_ROWS) return backward_s<E, SLAB, 8, CLUSTER>(a, s);
  return backward_s<E, SLAB, 4, CLUSTER>(a, s);
}

template <typename E>
cudaError_t backward_t(const RecurArgs &a, cudaStream_t s) {
  if constexpr (sizeof(E) == 2)
    if (wide(a.D) || (a.starts && a.B > MAX_SHORT_B))
      return wider(a.D) ? backward_w<E, 16, 8>(a, s) : backward_w<E, 16, 16>(a, s);
  return backward_w<E, 8, 16>(a, s);
}

}  // namespace

cudaError_t launch_recur_forward(const RecurArgs &a, cudaStream_t s) {
  return a.dtype == TWELL_BF16 ? forward_t<bf16>(a, s) : forward_t<float>(a, s);
}

cudaError_t launch_recur_backward(const RecurArgs &a, cudaStream_t s) {
  return a.dtype == TWELL_BF16 ? backward_t<bf16>(a, s) : backward_t<float>(a, s);
}

}  // namespace twell
