// Gated linear recurrence over a vector state (sm_100a): forward scan, its
// backward pass, and the one-token step.
//
//     h_t = a_t h_{t-1} + b_t,   a_t = exp(g_t),   b_t = x_t  or  (1 - a_t) x_t
//
// per channel, over sequences that follow each other on one token axis (a
// dense batch has a sequence start every T tokens, a packed one at cu[n]).
// The gradient carries c_t = dL/dh_t from the tokens after t:
//     d_t = dh_t + c_t,   c_{t-1} = a_t d_t      (c = dfinal at a sequence's end)
//     dx_t = d_t  or  (1 - a_t) d_t,   dg_t = a_t d_t (h_{t-1} [- x_t]),   dh_0 = a_1 d_1.
//
// Both directions are affine maps of the value that enters a span of tokens:
// (A, H) with out = A in + H.  What is carried from one group of 1024 or 2048 tokens to
// the next meets one rounded decay a group, exp of the sum of its g; within a group
// at most a warp's 16 or 32 tokens, three warps and fifteen tiles are joined by
// products of rounded ones.
// A span that holds a sequence start (an end, for the gradient) is "closed":
// what enters it does not reach what leaves it, whatever its value (an
// infinity or NaN of one sequence stays in it).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace gdr {
namespace {

constexpr int kCachedDevices = 64;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kWide = 64;         // channels of a tile, two a lane

// The two channels of a lane.  PAIRS: neighbours, rows and pointers aligned for
// it (and every row for tensor-map copies); else 32 apart, any alignment.
template <bool PAIRS> struct Lane {
  int c;         // the first channel
  bool on[2];    // which exist
  __device__ __forceinline__ Lane(int stripe, int D) {
    const int lane = threadIdx.x & 31;
    c = stripe * kWide + (PAIRS ? 2 * lane : lane);
    on[0] = c < D;
    on[1] = c + step() < D;
  }
  static __device__ __forceinline__ constexpr int step() { return PAIRS ? 1 : 32; }
  __device__ __forceinline__ bool any() const { return on[0]; }
};

// A lane's two channels.  Plain arithmetic: two chains of dependent product-sums
// that run side by side; the packed forms, which keep the pair in neighbouring
// registers, spilled here and were slower (177 against 189 us, 32768 x 4096
// bf16).  Long independent series (`fresh`) use them.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Two channels of one token as they are stored.
template <typename IO> struct Raw;
template <> struct Raw<float> {
  float2 r;
  __device__ __forceinline__ float2 value() const { return r; }
};
template <> struct Raw<__nv_bfloat16> {
  uint32_t r;
  __device__ __forceinline__ float2 value() const { return make_float2(bf16_lo(r), bf16_hi(r)); }
};

// Shared memory: a lane's two channels of a row.
template <bool PAIRS> __device__ __forceinline__ Raw<float> read_row(const float *row, int lane) {
  if constexpr (PAIRS) return {reinterpret_cast<const float2 *>(row)[lane]};
  else return {make_float2(row[lane], row[lane + 32])};
}
template <bool PAIRS> __device__ __forceinline__ Raw<__nv_bfloat16> read_row(const __nv_bfloat16 *row, int lane) {
  if constexpr (PAIRS) return {reinterpret_cast<const uint32_t *>(row)[lane]};
  const unsigned short *h = reinterpret_cast<const unsigned short *>(row);
  return {(uint32_t)h[lane] | (uint32_t)h[lane + 32] << 16};
}
template <bool PAIRS> __device__ __forceinline__ void write_row(float *row, int lane, float2 x) {
  if constexpr (PAIRS) {
    reinterpret_cast<float2 *>(row)[lane] = x;
  } else {
    row[lane] = x.x; row[lane + 32] = x.y;
  }
}

// Global memory: plain (coherent) accesses, states are updated in place by some calls.
template <bool PAIRS> __device__ __forceinline__ float2 load2(const float *p, const Lane<PAIRS> &l) {
  if constexpr (PAIRS) return *reinterpret_cast<const float2 *>(p + l.c);
  else return make_float2(p[l.c], l.on[1] ? p[l.c + 32] : 0.f);
}
template <bool PAIRS, typename IO> __device__ __forceinline__ void store2(IO *p, const Lane<PAIRS> &l, float2 x) {
  if constexpr (!PAIRS) {
    io<IO>::store(p + l.c, x.x);
    if (l.on[1]) io<IO>::store(p + l.c + 32, x.y);
  } else if constexpr (sizeof(IO) == 4) {
    *reinterpret_cast<float2 *>(p + l.c) = x;
  } else {
    *reinterpret_cast<uint32_t *>(p + l.c) = pack_bf16x2(x.x, x.y);
  }
}

// The decay of one token; for what enters from earlier tiles of the group, of a tile.
// With bf16 activations the fast exponential: off by 2^-22 of the value and, from
// the rounded product, 2^-24 |g|.  So much enters h before its rounding, and the fp32
// states, dg and dinitial_state (the accurate one changed their errors by less than
// a third, up as often as down, and cost 193 us instead of 180, 32768 x 4096).
template <typename IO> __device__ __forceinline__ float2 decay(float2 g) {
  if constexpr (sizeof(IO) == 2) {
    const float2 t = mul2(g, both(1.44269504f));  // log2 e
    float2 a;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a.y) : "f"(t.y));
    return a;
  } else {
    return make_float2(expf(g.x), expf(g.y));
  }
}
// 1 - a of one token: near 0 the series of -expm1(g), whose first term left out
// is below 2^-21.9 of the value (bf16 activations) or 2^-30, else the difference,
// which then loses less than two bits.
template <typename IO> __device__ __forceinline__ float2 fresh(float2 g, float2 a) {
  float2 s = both(1.f / 5040.f);
  if constexpr (sizeof(IO) == 4) {
    s = both(1.f / 362880.f);
    s = __ffma2_rn(s, g, both(1.f / 40320.f));
    s = __ffma2_rn(s, g, both(1.f / 5040.f));
  }
  s = __ffma2_rn(s, g, both(1.f / 720.f));
  s = __ffma2_rn(s, g, both(1.f / 120.f));
  s = __ffma2_rn(s, g, both(1.f / 24.f));
  s = __ffma2_rn(s, g, both(1.f / 6.f));
  s = __ffma2_rn(s, g, both(0.5f));
  s = __ffma2_rn(s, g, both(1.f));
  const float2 near = mul2(make_float2(-g.x, -g.y), s), far = fma2(a, both(-1.f), both(1.f));
  return make_float2(g.x > -0.5f ? near.x : far.x, g.y > -0.5f ? near.y : far.y);
}
// What a token adds to the state: x, or (1 - a) x.
template <typename IO, bool COMPLEMENT> __device__ __forceinline__ float2 input(float2 g, float2 a, float2 x) {
  if constexpr (COMPLEMENT) return mul2(fresh<IO>(g, a), x);
  else return x;
}

// Row of sequence n's state in the states or the pool, or -1 (no slot).
__device__ __forceinline__ int state_row(const GlrArgs &p, int n) {
  if (!p.state_slots) return n;
  const int s = __ldg(p.state_slots + n);
  return s >= 0 && s < p.num_slots ? s : -1;
}

// Which of a warp's TOK tokens begin or end a sequence (bit i: token t0 + i), and,
// in lane i where token t0 + i does, the row of that sequence's states (or -1).
struct Marks {
  uint32_t first, last;
  int row;
  __device__ __forceinline__ int row_of(int i) const { return __shfl_sync(0xffffffffu, row, i); }
  // Whether one begins behind the first token, or ends before the last.  Those
  // that begin and end with the warp's tokens (sequences of whole warps) take the
  // path without marks.
  template <int TOK> __device__ __forceinline__ bool inside() const {
    return (first & ~1u) | (last & ~(1u << (TOK - 1)));
  }
};
template <int TOK> __device__ __forceinline__ Marks find_marks(const GlrArgs &p, uint32_t t0, int lane) {
  static_assert(TOK <= 32, "a lane a token");
  Marks m;
  bool f = false, l = false;
  m.row = -1;
  const uint32_t t = t0 + lane;
  if (lane < TOK && t < (uint32_t)p.tokens) {
    int seq;
    if (p.cu_seqlens) {  // the last sequence that starts at or before t (empty ones start there too)
      int lo = 0, hi = p.num_seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((uint32_t)__ldg(p.cu_seqlens + mid) <= t) lo = mid;
        else hi = mid;
      }
      seq = lo;
      f = (uint32_t)__ldg(p.cu_seqlens + lo) == t;
      l = (uint32_t)__ldg(p.cu_seqlens + lo + 1) == t + 1;
    } else {
      seq = (int)(t / (uint32_t)p.T);
      const uint32_t r = t - (uint32_t)seq * (uint32_t)p.T;
      f = r == 0;
      l = r == (uint32_t)p.T - 1;
    }
    if ((f || l) && GDR_IN_BOUNDS(seq < p.num_seqs)) m.row = state_row(p, seq);
  }
  m.first = __ballot_sync(0xffffffffu, f);
  m.last = __ballot_sync(0xffffffffu, l);
  return m;
}

// Row `r` of a [rows, D] array of states; zeros where there is none.
template <bool PAIRS>
__device__ __forceinline__ float2 load_row(const GlrArgs &p, const float *states, int r, const Lane<PAIRS> &l) {
  return states && l.any() && r >= 0 && GDR_IN_BOUNDS(r < p.num_slots) ? load2<PAIRS>(states + (int64_t)r * p.D, l) : both(0.f);
}
template <bool PAIRS>
__device__ __forceinline__ void store_state(const GlrArgs &p, float *states, int r, const Lane<PAIRS> &l, float2 x) {
  if (states && l.any() && r >= 0 && GDR_IN_BOUNDS(r < p.num_slots)) store2<PAIRS>(states + (int64_t)r * p.D, l, x);
}

// Whether the call has failed before this kernel: bad offsets, or a wait of its
// first pass that gave up.
__device__ __forceinline__ bool failed(const GlrArgs &p) {
  return (p.cu_seqlens || p.keep_status) && *reinterpret_cast<const volatile int32_t *>(p.status) != KDA_DEVICE_OK;
}

// ---- maps of spans ------------------------------------------------------
// A span of tokens takes what enters it, `in`, to A in + H, or to H where it is
// closed: A = -1 (a decay is never below 0).  All channels of a span are closed
// or none.
struct Map2 {  // of a lane's two channels
  float2 A, H;
  __device__ __forceinline__ bool closed() const { return A.x < 0.f; }
  __device__ __forceinline__ float2 of(float2 in) const {
    const float2 t = fma2(A, in, H);
    return closed() ? H : t;
  }
};
constexpr float kClosed = -1.f;
// The map of n spans one after the other.
template <int N> __device__ __forceinline__ Map2 joined(const Map2 (&t)[N]) {
  Map2 m = t[0];
  bool closed = false;
#pragma unroll
  for (int j = 0; j < N; ++j) closed |= t[j].closed();
  if (!closed) {
#pragma unroll
    for (int j = 1; j < N; ++j) {
      m.H = fma2(t[j].A, m.H, t[j].H);
      m.A = mul2(m.A, t[j].A);
    }
  } else {
#pragma unroll
    for (int j = 1; j < N; ++j) m.H = t[j].of(m.H);
    m.A = both(kClosed);
  }
  return m;
}

struct TileShared {
  // the warps' maps and the sums of their log-decays; a tile's are read until its
  // end, while the next one's are written
  Map2 map[2][kWarps][32];
  float2 sum[2][kWarps][32];
  Map2 before[kWarps][32];  // of earlier tiles, a part a warp
  float2 before_sum[kWarps][32];
  uint64_t full[kWarps];    // a warp's copies have landed
  uint32_t step;            // of the block's next tile
  int stripe;
};

// ---- the chain of tiles -------------------------------------------------
// Blocks take tiles in order of a ticket, each its own in rising order, so
// every tile that another waits for is done or in the hands of a block that
// waits for earlier ones only: the lowest open ticket always proceeds.  In
// groups of tiles a tile publishes its map as soon as it has it; what
// enters a tile is what enters its group, through the maps of the group's tiles
// before it; the last tile of a group publishes what leaves the group.  Which
// values are joined, and in which order, depends on the sizes alone, never on
// timing.
//
// A group's decay is exp of the sum of its log-decays, not the product of its tiles'
// decays: only what a group hands on is carried from group to group, and rounded
// factors that are all alike err to the same side.  (Decays of 1e-5 a token, constant
// over 32768: h off by 8e-7 of itself in fp32, by products of the warps' decays
// 2.4e-5.  It costs bf16 1 % of its time.)
//
// A channel's map goes through the workspace as one 64-bit word (the bits of the
// sum turned above, H below), which is its own flag: 0 is not there yet, and no map
// is 0.  A closed map has a pattern of its own: that of a NaN which no sum gives (sums
// that are not numbers have one pattern, 0x7fffffff).  So a hand-over is one store and
// one polling load, without a fence.  The rows of words are as wide as the tiles
// (`pitch`), so every lane has its own.
template <int TOK> struct Chain {
  static constexpr int kGroup = kGlrGroup, kPart = kGroup / kWarps;
  static_assert(kGroup >= kGlrShortestGroup, "the workspace counts groups of at least this length");
};
struct Words {
  uint64_t u[2];
  __device__ __forceinline__ bool here() const { return min((uint32_t)(u[0] >> 32), (uint32_t)(u[1] >> 32)) != 0; }
  static constexpr uint32_t kClosedSum = 0x7ffffffeu;
  static __device__ __forceinline__ uint64_t pack(bool closed, float sum, float H) {
    return (uint64_t)max(~(closed ? kClosedSum : __float_as_uint(sum)), 1u) << 32 | __float_as_uint(H);
  }
  static __device__ __forceinline__ uint32_t above(uint64_t u) { return ~(uint32_t)(u >> 32); }
  __device__ __forceinline__ bool closed() const { return above(u[0]) == kClosedSum; }
  __device__ __forceinline__ float2 sum() const {
    return make_float2(__uint_as_float(above(u[0])), __uint_as_float(above(u[1])));
  }
  __device__ __forceinline__ float2 H() const {
    return make_float2(__uint_as_float((uint32_t)u[0]), __uint_as_float((uint32_t)u[1]));
  }
};
template <bool PAIRS> __device__ __forceinline__ void load_words(const uint64_t *p, Words &w) {
  if constexpr (PAIRS) {
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(w.u[0]), "=l"(w.u[1]) : "l"(p) : "memory");
  } else {
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w.u[0]) : "l"(p) : "memory");
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w.u[1]) : "l"(p + 32) : "memory");
  }
}
template <bool PAIRS> __device__ __forceinline__ void store_words(uint64_t *p, bool closed, float2 sum, float2 H) {
  const uint64_t u[2] = {Words::pack(closed, sum.x, H.x), Words::pack(closed, sum.y, H.y)};
  if constexpr (PAIRS) {
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p), "l"(u[0]), "l"(u[1]) : "memory");
  } else {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(u[0]) : "memory");
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p + 32), "l"(u[1]) : "memory");
  }
}

// A tile's place in the chain (REV: from the last tile on).
struct Place {
  uint32_t step, tile;
  int stripe;
};

// Takes the block's next tile (one thread).  Without a chain: `grid` tiles on.
__device__ __forceinline__ uint32_t next_ticket(const GlrArgs &p, TileShared &sh, uint32_t last) {
  const uint32_t t = p.chained ? (uint32_t)atomicAdd(p.ticket, 1) : last + gridDim.x;
  sh.step = t / (uint32_t)p.stripes;
  sh.stripe = (int)(t - sh.step * (uint32_t)p.stripes);
  return t;
}
template <bool REV> __device__ __forceinline__ Place taken(const GlrArgs &p, const TileShared &sh) {
  Place q;
  q.step = sh.step;
  q.stripe = sh.stripe;
  q.tile = REV ? (uint32_t)p.tiles - 1 - q.step : q.step;
  return q;
}

// Whether a wait gives up (here, or elsewhere: the status word says so).
__device__ __forceinline__ bool give_up(const GlrArgs &p, uint32_t poll) {
  if ((poll & 1023) != 1023) return false;
  if (*reinterpret_cast<const volatile int32_t *>(p.status) != KDA_DEVICE_OK) return true;
  if (poll < p.max_polls) return false;
  *p.status = KDA_DEVICE_TIMEOUT;
  return true;
}

// After the warps have shared their maps, one of them publishes the tile's,
// unless the tile ends its group.
template <bool PAIRS, bool REV>
__device__ __forceinline__ void publish_tile(const GlrArgs &p, const TileShared &sh, int buf, const Place &q,
                                             int c, int lane) {
  Map2 t[kWarps];
  float2 sum = both(0.f);
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    t[k] = sh.map[buf][REV ? kWarps - 1 - k : k][lane];
    sum = add2(sum, sh.sum[buf][REV ? kWarps - 1 - k : k][lane]);
  }
  const Map2 m = joined(t);
  if (GDR_IN_BOUNDS(q.step < p.tiles && c < p.pitch))
    store_words<PAIRS>(p.tile_map + (int64_t)q.step * p.pitch + c, m.closed(), sum, m.H);
}

// What enters the tile.  Each warp joins its part of the group's earlier maps,
// then all wait for what enters the group and take it through the parts.  That
// wait is the serial part of the chain: the tile that ends a group has the whole
// group's map ready and sends on what leaves it at once.  Every thread of the block
// takes part.  False: a wait gave up.
template <typename IO, int TOK, bool PAIRS, bool REV>
__device__ __forceinline__ bool enter_tile(const GlrArgs &p, TileShared &sh, int buf, const Place &q, int c, int w,
                                           int lane, float2 &in) {
  constexpr int kGroup = Chain<TOK>::kGroup, kPart = Chain<TOK>::kPart;
  const uint32_t group = q.step / kGroup;
  const int at = q.step % kGroup, n = at - w * kPart;  // maps to join (at most kPart)
  bool ok = true;
  // (the carry of a group begun long ago is there by now, or looked at again below)
  const bool behind = q.step >= kGroup && GDR_IN_BOUNDS(group <= p.groups && c < p.pitch);
  const uint64_t *carry = p.carry + ((int64_t)group - 1) * p.pitch + c;
  Words u;
  u.u[0] = u.u[1] = 0;
  if (behind) load_words<PAIRS>(carry, u);
  if (n > 0 && GDR_IN_BOUNDS(q.step < p.tiles && c < p.pitch)) {
    const uint64_t *from = p.tile_map + (int64_t)(q.step - n) * p.pitch + c;
    Words t[kPart];
#pragma unroll
    for (int j = 0; j < kPart; ++j) {
      t[j].u[0] = t[j].u[1] = Words::pack(false, 0.f, 0.f);  // nothing changes
      if (j < n) load_words<PAIRS>(from + (int64_t)j * p.pitch, t[j]);
    }
    for (uint32_t poll = 0;; ++poll) {
      bool have = true;
#pragma unroll
      for (int j = 0; j < kPart; ++j) have = have && t[j].here();
      if (__all_sync(0xffffffffu, have)) break;
      if (give_up(p, poll)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int j = 0; j < kPart; ++j)
        if (!t[j].here()) load_words<PAIRS>(from + (int64_t)j * p.pitch, t[j]);
    }
    Map2 m[kPart];
    float2 sum = both(0.f);
#pragma unroll
    for (int j = 0; j < kPart; ++j) {
      m[j] = {t[j].closed() ? both(kClosed) : decay<IO>(t[j].sum()), t[j].H()};
      sum = add2(sum, t[j].sum());
    }
    sh.before[w][lane] = joined(m);
    sh.before_sum[w][lane] = sum;
  }
  if (__syncthreads_or(!ok)) return false;
  Map2 pre = {both(1.f), both(0.f)};  // of the group's tiles before this one
#pragma unroll
  for (int k = 0; k < kWarps; ++k)
    if (k * kPart < at) {
      const Map2 t = sh.before[k][lane];
      pre = {pre.closed() || t.closed() ? both(kClosed) : mul2(pre.A, t.A), t.of(pre.H)};
    }
  // and of the whole group, by the warp that sends on what leaves it
  const bool ends = at == kGroup - 1 && w == (REV ? 0 : kWarps - 1);
  Map2 all = pre;
  if (ends) {
    float2 sum = both(0.f);
    bool shut = pre.closed();
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const Map2 t = sh.map[buf][REV ? kWarps - 1 - k : k][lane];
      all.H = t.of(all.H);
      shut |= t.closed();
      sum = add2(sum, add2(sh.before_sum[k][lane], sh.sum[buf][k][lane]));
    }
    all.A = shut ? both(kClosed) : make_float2(expf(sum.x), expf(sum.y));
  }
  in = both(0.f);
  if (behind && !pre.closed()) {  // (nothing to wait for where a sequence began since)
    for (uint32_t poll = 0; !__all_sync(0xffffffffu, u.here()); ++poll) {
      if (give_up(p, poll)) {
        ok = false;  // the block finds out at its next barrier
        break;
      }
      load_words<PAIRS>(carry, u);
    }
    in = u.H();
  }
  if (ok && ends && GDR_IN_BOUNDS(group < p.groups && c < p.pitch))
    store_words<PAIRS>(p.carry + (int64_t)group * p.pitch + c, true, both(0.f), all.of(in));
  in = pre.of(in);
  return ok;
}

// `x`, what enters the tile, becomes what enters warp w.
template <bool REV>
__device__ __forceinline__ void enter_warp(const Map2 (&map)[kWarps][32], int w, int lane, float2 &x) {
#pragma unroll
  for (int k = 0; k < kWarps - 1; ++k) {
    const int j = REV ? kWarps - 1 - k : k;
    if (REV ? j > w : j < w) x = map[j][lane].of(x);
  }
}

// Sequences without tokens, by the blocks of the first tile: what leaves them
// is what enters them.
__device__ __forceinline__ void pass_empty(const GlrArgs &p, const float *src, float *dst, bool pooled,
                                           int c0, int width) {
  if (!dst || !p.cu_seqlens) return;
  const int lane = threadIdx.x & 31;
  for (int n0 = (threadIdx.x >> 5) * 32; n0 < p.num_seqs; n0 += kThreads) {
    const int n = n0 + lane;
    const bool empty = n < p.num_seqs && __ldg(p.cu_seqlens + n) == __ldg(p.cu_seqlens + n + 1);
    uint32_t todo = __ballot_sync(0xffffffffu, empty);
    while (todo) {
      const int k = n0 + __ffs(todo) - 1;
      todo &= todo - 1;
      const int64_t r = pooled ? state_row(p, k) : k;
      if (r < 0) continue;
      for (int c = c0 + lane; c < c0 + width && c < p.D; c += 32)
        dst[r * p.D + c] = src ? src[r * p.D + c] : 0.f;
    }
  }
}

// Whether a tile holds the start or the end of a sequence (else its tokens take
// the path without marks).  (A plain load: the kernel that writes the marks may
// still run when this one starts, so they are not read-only to it.)
__device__ __forceinline__ bool has_marks(const GlrArgs &p, uint32_t tile) {
  if (p.cu_seqlens) return p.tile_marks[tile] != 0;
  const uint32_t t = tile * p.tile_tokens, r = t % (uint32_t)p.T;
  return r == 0 || r + p.tile_tokens >= (uint32_t)p.T;
}

// ---- the kernels --------------------------------------------------------
// Persistent blocks of four warps; a tile is TOK tokens a warp and 64 channels.
// Each warp copies its own rows to shared memory (tensor-map copies) and waits
// for them alone.  In the
// first pass over a tile its rows go to registers, so that the next tile's
// copies run while this one waits for what enters it and is written: one read
// of each input.  What an SM moves is what its blocks hold (registers and the
// copies under way) over the time a tile takes, two or three L2 round trips.
//
// A warp with a sequence start or end inside its tokens takes rolled loops instead,
// over the rows in shared memory, and its next copies begin after them (256
// sequences of 64 x 4096 bf16, all of whole warps: 83 us; by rolled loops 127).
//
// Bound by HBM where rows are long (32768 x 4096: bf16 174 us = 6.2 TB/s of 2e + 4
// bytes an element, fp32 253 us = 6.4; a copy does 6.5), with few columns by the
// chain (65536 x 256 bf16: 40 us = 3.4 TB/s).  The complement forms 1 - a, 8 warps
// an SM (bf16 237 us, fp32 267).
//
// A tensor-map copy begins on 16 bytes.  Where rows do not, every R-th one (R
// elements in 16 bytes) is as far past a boundary as the first: R maps, each of
// every R-th row and from the boundary before it, reach them all, and lanes read
// `shift` elements on.  (By lane copies of 4 or 2 bytes instead: 431 us against
// 275 for 32767 x 4095 fp32, 347 against 239 for bf16.)
struct Shift {  // of row i, where the first token's is s: s + i l
  int s, l;
};
template <typename T> __device__ __forceinline__ Shift shift_of(const void *base, int64_t ld) {
  constexpr int R = 16 / sizeof(T);
  return {(int)(reinterpret_cast<uintptr_t>(base) / sizeof(T) % R), (int)(ld % R)};
}
// A warp's rows of one tensor in shared memory.
template <typename T, int TOK, bool PAIRS> struct alignas(128) TensorRows {
  static constexpr int R = PAIRS ? 1 : 16 / sizeof(T), kPitch = kWide + (PAIRS ? 0 : R);
  static constexpr int kBox = TOK / R * kPitch * (int)sizeof(T), kBytes = R * kBox;  // a copy, and all
  static_assert(TOK % R == 0, "the same row of every warp has the same shift");
  T v[R][(kBox + 127) / 128 * 128 / sizeof(T)];
  __device__ __forceinline__ T *row(int i, Shift q) {
    return v[i % R] + i / R * kPitch + (PAIRS ? 0 : (q.s + i * q.l) & (R - 1));
  }
};
template <typename IO, bool PAIRS, int TOK, bool BWD> struct WarpRows {
  TensorRows<float, TOK, PAIRS> g;
  TensorRows<IO, TOK, PAIRS> x;
  static constexpr int kBytes = decltype(g)::kBytes + decltype(x)::kBytes;
};
template <typename IO, bool PAIRS, int TOK> struct WarpRows<IO, PAIRS, TOK, true> {
  TensorRows<float, TOK, PAIRS> g;
  TensorRows<IO, TOK, PAIRS> x, dh;
  static constexpr int kBytes = decltype(g)::kBytes + 2 * decltype(x)::kBytes;
};
template <typename IO, bool PAIRS, bool BWD> struct GlrMaps {
  static constexpr int kIO = PAIRS ? 1 : 16 / sizeof(IO), kF = PAIRS ? 1 : 4;
  CUtensorMap g[kF], x[kIO], dh[BWD ? kIO : 1];
};

// Tokens of a warp that exist.
template <int TOK> __device__ __forceinline__ int tokens_of(const GlrArgs &p, uint32_t t0) {
  const int64_t left = p.tokens - (int64_t)t0;
  return left <= 0 ? 0 : left < TOK ? (int)left : TOK;
}

// Begins the copies of a warp's rows of a tile.
template <typename IO, bool PAIRS, int TOK, bool BWD>
__device__ __forceinline__ void begin_copies(const GlrMaps<IO, PAIRS, BWD> &maps, WarpRows<IO, PAIRS, TOK, BWD> &rows,
                                             uint64_t *full, const Place &q, int w, int lane) {
  using Maps = GlrMaps<IO, PAIRS, BWD>;
  const int t0 = (int)(q.tile * (kWarps * TOK) + w * TOK), c0 = q.stripe * kWide;
  __syncwarp();  // the rows have been read by every lane
  if (lane == 0) tc::mbar_arrive_expect_tx(full, rows.kBytes);
  if (!PAIRS) __syncwarp();
  if (lane < Maps::kF) tc::tma_load_2d(rows.g.v[lane], &maps.g[lane], c0, t0 / Maps::kF, full);
  if (lane < Maps::kIO) {
    tc::tma_load_2d(rows.x.v[lane], &maps.x[lane], c0, t0 / Maps::kIO, full);
    if constexpr (BWD) tc::tma_load_2d(rows.dh.v[lane], &maps.dh[lane], c0, t0 / Maps::kIO, full);
  }
}
__device__ __forceinline__ bool copies_done(const GlrArgs &p, uint64_t *full, uint32_t parity) {
  return tc::mbar_wait_warp(full, parity, p.status, KDA_DEVICE_TIMEOUT);
}
__device__ __forceinline__ void init_barriers(TileShared &sh) {
  if (threadIdx.x < kWarps) tc::mbar_init(&sh.full[threadIdx.x], 1);
  tc::mbar_fence_init();
}

// Tokens a warp, and blocks an SM by their registers.  The chain and the barriers
// cost about as much for a long tile as for a short one, so a tile is as long as
// the registers allow: forward in bf16, 32 tokens a warp (a and the packed x in 96
// registers, three blocks), else 16 (four blocks).
template <typename IO, bool PAIRS, bool COMPLEMENT> struct FwdShape {
  static constexpr bool kLong = PAIRS && sizeof(IO) == 2;
  static constexpr int kTok = kLong ? 32 : 16, kBlocks = kLong ? COMPLEMENT ? 2 : 3 : 4;
};
// Backward: in bf16 x and dh go to registers as well; else (x and dh too wide, or
// g needed again) they are read from shared memory in both passes, and the next
// copies begin after the second.  Three blocks also in fp32, whose tiles leave room
// for no more (with the registers of four: 459 and 529 us against 453 and 502).
template <typename IO, bool COMPLEMENT> struct BwdShape {
  static constexpr bool kEarly = sizeof(IO) == 2 && !COMPLEMENT;
  static constexpr int kTok = 16, kBlocks = kEarly || sizeof(IO) == 4 ? 3 : 4;
};

// Forward.  STATES_ONLY: only the saved chunk states are written.
template <typename IO, bool PAIRS, bool COMPLEMENT, bool STATES_ONLY>
__global__ void __launch_bounds__(kThreads, (FwdShape<IO, PAIRS, COMPLEMENT>::kBlocks))
glr_scan_kernel(const __grid_constant__ GlrArgs p, const __grid_constant__ GlrMaps<IO, PAIRS, false> maps) {
  constexpr int TOK = FwdShape<IO, PAIRS, COMPLEMENT>::kTok;
  __shared__ TileShared sh;
  __shared__ float2 start[kWarps][32];  // a state that a warp's tokens begin with
  extern __shared__ __align__(128) unsigned char tile_bytes[];
  init_barriers(sh);
  wait_for_last();
  if (failed(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  auto &rows = reinterpret_cast<WarpRows<IO, PAIRS, TOK, false> *>(tile_bytes)[w];
  const Shift sg = shift_of<float>(p.g, p.ld_g), sx = shift_of<IO>(p.x, p.ld_x);
  uint32_t ticket = 0, parity = 0;
  if (threadIdx.x == 0) ticket = next_ticket(p, sh, blockIdx.x - gridDim.x);
  __syncthreads();
  Place q = taken<false>(p, sh);
  if (q.step >= p.tiles) return;
  __syncthreads();
  begin_copies(maps, rows, &sh.full[w], q, w, lane);
  bool marked = has_marks(p, q.tile), alive = true;
  while (true) {
    if (threadIdx.x == 0) ticket = next_ticket(p, sh, ticket);
    Lane<PAIRS> l(q.stripe, p.D);
    const uint32_t t0 = q.tile * (kWarps * TOK) + w * TOK;
    Marks m;
    m.first = m.last = 0;
    m.row = -1;
    if (marked) m = find_marks<TOK>(p, t0, lane);
    const bool inside = m.inside<TOK>();
    alive &= copies_done(p, &sh.full[w], parity);
    const int buf = parity;
    parity ^= 1;
    // the map of the warp's tokens
    float2 a[TOK], b[COMPLEMENT ? TOK : 1], gs = both(0.f), h = both(0.f);
    Raw<IO> x[COMPLEMENT ? 1 : TOK];
    auto b_of = [&](int i) { return COMPLEMENT ? b[COMPLEMENT ? i : 0] : x[COMPLEMENT ? 0 : i].value(); };
    auto g_row = [&](int i) { return read_row<PAIRS>(rows.g.row(i, sg), lane).value(); };
    auto rolled = [&](int i, float2 g, float2 y) {  // the state after y by token i
      const float2 ai = decay<IO>(g);
      return fma2(ai, y, input<IO, COMPLEMENT>(g, ai, read_row<PAIRS>(rows.x.row(i, sx), lane).value()));
    };
    // An initial state is read once, before the map is published: the sequence's
    // last tile may write the final state over it as soon as that is done.
    if (!inside) {
      if (m.first) start[w][lane] = h = load_row<PAIRS>(p, p.initial_state, m.row_of(0), l);
#pragma unroll
      for (int i = 0; i < TOK; ++i) {
        const float2 g = g_row(i);
        const Raw<IO> xi = read_row<PAIRS>(rows.x.row(i, sx), lane);
        a[i] = decay<IO>(g);
        if (COMPLEMENT) b[COMPLEMENT ? i : 0] = input<IO, COMPLEMENT>(g, a[i], xi.value());
        else x[COMPLEMENT ? 0 : i] = xi;
        gs = add2(gs, g);
      }
#pragma unroll
      for (int i = 0; i < TOK; ++i) h = fma2(a[i], h, b_of(i));
    } else {
      // The state after a start takes the place of its g.  Four at a time.
      for (uint32_t todo = m.first; todo;) {
        int at[4];
        float2 h0[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          at[k] = __ffs(todo) - 1;
          todo &= todo - 1;
          if (at[k] >= 0) h0[k] = load_row<PAIRS>(p, p.initial_state, m.row_of(at[k]), l);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at[k] >= 0) write_row<PAIRS>(rows.g.row(at[k], sg), lane, rolled(at[k], g_row(at[k]), h0[k]));
      }
#pragma unroll 4
      for (int i = 0; i < TOK; ++i) {
        const float2 g = g_row(i), t = rolled(i, g, h);
        h = m.first >> i & 1 ? g : t;
        gs = add2(gs, g);  // (of no use in a closed span)
      }
    }
    sh.map[buf][w][lane] = {m.first ? both(kClosed) : make_float2(expf(gs.x), expf(gs.y)), h};
    sh.sum[buf][w][lane] = gs;
    if (__syncthreads_or(!alive)) return;  // a wait gave up; no copy is under way
    if (p.chained && w == kWarps - 1 && (q.step + 1) % Chain<TOK>::kGroup != 0) publish_tile<PAIRS, false>(p, sh, buf, q, l.c, lane);
    const Place nq = taken<false>(p, sh);
    const bool more = nq.step < p.tiles;
    if (more && !inside) begin_copies(maps, rows, &sh.full[w], nq, w, lane);
    const bool next_marked = more && has_marks(p, nq.tile);
    h = both(0.f);
    if (p.chained) {
      alive = enter_tile<IO, TOK, PAIRS, false>(p, sh, buf, q, l.c, w, lane, h);
      if (!alive) l.on[0] = l.on[1] = false;  // writes nothing, and ends at the next barrier
    } else {
      __syncthreads();  // the next ticket is read before it is replaced
    }
    enter_warp<false>(sh.map[buf], w, lane, h);
    // (a chunk's first token is a warp's)
    if (p.chunk_states && t0 % kGlrChunk == 0 && l.any() && t0 < p.tokens && GDR_IN_BOUNDS(t0 / kGlrChunk < p.chunks))
      store2<PAIRS>(p.chunk_states + (int64_t)(t0 / kGlrChunk) * p.D, l, h);
    if (!STATES_ONLY) {
      IO *out = static_cast<IO *>(p.h) + (int64_t)t0 * p.D;
      const int n = l.any() ? tokens_of<TOK>(p, t0) : 0;
      if (!inside) {
        if (m.first) h = start[w][lane];
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
          h = fma2(a[i], h, b_of(i));
          if (i < n && GDR_IN_BOUNDS((int64_t)t0 + i < p.tokens)) store2<PAIRS>(out + (int64_t)i * p.D, l, h);
        }
        if (m.last) store_state<PAIRS>(p, p.final_state, m.row_of(TOK - 1), l, h);
      } else {
#pragma unroll 4
        for (int i = 0; i < TOK; ++i) {
          const float2 g = g_row(i), t = rolled(i, g, h);
          h = m.first >> i & 1 ? g : t;
          if (i < n && GDR_IN_BOUNDS((int64_t)t0 + i < p.tokens)) store2<PAIRS>(out + (int64_t)i * p.D, l, h);
          if (m.last >> i & 1) store_state<PAIRS>(p, p.final_state, m.row_of(i), l, h);
        }
      }
      if (q.tile == 0) pass_empty(p, p.initial_state, p.final_state, true, q.stripe * kWide, kWide);
    }
    if (!more) return;
    if (inside) {
      tc::fence_async_smem();  // states were written over rows of g
      begin_copies(maps, rows, &sh.full[w], nq, w, lane);
    }
    marked = next_marked;
    q = nq;
  }
}

// Backward: the states again from what enters the tile (saved), the gradients
// from what enters it from the tokens after it (chained).  32768 x 4096: bf16 324
// us = 5.8 TB/s of 3e + 8 bytes an element, fp32 443 us = 6.1; complement 372, 490.
template <typename IO, bool PAIRS, bool COMPLEMENT>
__global__ void __launch_bounds__(kThreads, (BwdShape<IO, COMPLEMENT>::kBlocks))
glr_gradient_kernel(const __grid_constant__ GlrArgs p, const __grid_constant__ GlrMaps<IO, PAIRS, true> maps) {
  constexpr bool EARLY = BwdShape<IO, COMPLEMENT>::kEarly;
  constexpr int TOK = BwdShape<IO, COMPLEMENT>::kTok;
  static_assert(kWarps * TOK == kGlrChunk, "a tile is a chunk: its saved state enters it");
  __shared__ TileShared sh;
  __shared__ Map2 states[kWarps][32];  // the warps' maps of the states
  extern __shared__ __align__(128) unsigned char tile_bytes[];
  init_barriers(sh);
  wait_for_last();
  if (failed(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  auto &rows = reinterpret_cast<WarpRows<IO, PAIRS, TOK, true> *>(tile_bytes)[w];
  const Shift sg = shift_of<float>(p.g, p.ld_g), sx = shift_of<IO>(p.x, p.ld_x), sd = shift_of<IO>(p.dh, p.ld_dh);
  uint32_t ticket = 0, parity = 0;
  if (threadIdx.x == 0) ticket = next_ticket(p, sh, blockIdx.x - gridDim.x);
  __syncthreads();
  Place q = taken<true>(p, sh);
  if (q.step >= p.tiles) return;
  __syncthreads();
  begin_copies(maps, rows, &sh.full[w], q, w, lane);
  bool marked = has_marks(p, q.tile), alive = true;
  while (true) {
    if (threadIdx.x == 0) ticket = next_ticket(p, sh, ticket);
    Lane<PAIRS> l(q.stripe, p.D);
    const uint32_t t0 = q.tile * (kWarps * TOK) + w * TOK;
    float2 h = both(0.f), s = both(0.f), r = both(0.f), gs = both(0.f);
    if (l.any() && GDR_IN_BOUNDS(q.tile < p.chunks)) h = load2<PAIRS>(p.chunk_states + (int64_t)q.tile * p.D, l);
    Marks m;
    m.first = m.last = 0;
    m.row = -1;
    if (marked) m = find_marks<TOK>(p, t0, lane);
    const bool inside = m.inside<TOK>();
    alive &= copies_done(p, &sh.full[w], parity);
    const int buf = parity;
    parity ^= 1;
    float2 a[TOK];
    Raw<IO> xk[EARLY ? TOK : 1], dk[EARLY ? TOK : 1];
    auto g_row = [&](int i) { return read_row<PAIRS>(rows.g.row(i, sg), lane).value(); };
    auto x_row = [&](int i) { return read_row<PAIRS>(rows.x.row(i, sx), lane).value(); };
    auto d_row = [&](int i) { return read_row<PAIRS>(rows.dh.row(i, sd), lane).value(); };
    auto x_of = [&](int i) { return EARLY ? xk[EARLY ? i : 0].value() : x_row(i); };
    auto d_of = [&](int i) { return EARLY ? dk[EARLY ? i : 0].value() : d_row(i); };
    // the state after y by token i
    auto advance = [&](int i, float2 x, float2 y) {
      return fma2(a[i], y, COMPLEMENT ? input<IO, COMPLEMENT>(g_row(i), a[i], x) : x);
    };
    auto rolled = [&](int i, float2 y) {
      const float2 g = g_row(i), ai = decay<IO>(g);
      return fma2(ai, y, input<IO, COMPLEMENT>(g, ai, x_row(i)));
    };
    if (!inside) {
      if (m.first) s = load_row<PAIRS>(p, p.initial_state, m.row_of(0), l);
      if (m.last) r = load_row<PAIRS>(p, p.dfinal, m.row_of(TOK - 1), l);
#pragma unroll
      for (int i = 0; i < TOK; ++i) {
        const float2 g = g_row(i);
        if (EARLY) {
          xk[EARLY ? i : 0] = read_row<PAIRS>(rows.x.row(i, sx), lane);
          dk[EARLY ? i : 0] = read_row<PAIRS>(rows.dh.row(i, sd), lane);
        }
        a[i] = decay<IO>(g);
        gs = add2(gs, g);
      }
#pragma unroll
      for (int i = 0; i < TOK; ++i) s = advance(i, x_of(i), s);
#pragma unroll
      for (int i = TOK - 1; i >= 0; --i) r = mul2(a[i], add2(d_of(i), r));
    } else {
#pragma unroll 2
      for (int i = 0; i < TOK; ++i) {
        if (m.first >> i & 1) s = load_row<PAIRS>(p, p.initial_state, m.row_of(i), l);
        s = rolled(i, s);
        gs = add2(gs, g_row(i));
      }
#pragma unroll 2
      for (int i = TOK - 1; i >= 0; --i) {  // the end of a sequence brings its final state's gradient
        if (m.last >> i & 1) r = load_row<PAIRS>(p, p.dfinal, m.row_of(i), l);
        r = mul2(decay<IO>(g_row(i)), add2(d_row(i), r));
      }
    }
    {
      const float2 A = make_float2(expf(gs.x), expf(gs.y));
      sh.map[buf][w][lane] = {m.last ? both(kClosed) : A, r};
      sh.sum[buf][w][lane] = gs;
      states[w][lane] = {m.first ? both(kClosed) : A, s};
    }
    if (__syncthreads_or(!alive)) return;  // a wait gave up; no copy is under way
    if (p.chained && w == 0 && (q.step + 1) % Chain<TOK>::kGroup != 0) publish_tile<PAIRS, true>(p, sh, buf, q, l.c, lane);
    const Place nq = taken<true>(p, sh);
    const bool more = nq.step < p.tiles;
    if (EARLY && more && !inside) begin_copies(maps, rows, &sh.full[w], nq, w, lane);
    const bool next_marked = more && has_marks(p, nq.tile);
    enter_warp<false>(states, w, lane, h);
    r = both(0.f);
    if (p.chained) {
      alive = enter_tile<IO, TOK, PAIRS, true>(p, sh, buf, q, l.c, w, lane, r);
      if (!alive) l.on[0] = l.on[1] = false;  // writes nothing, and ends at the next barrier
    } else {
      __syncthreads();  // the next ticket is read before it is replaced
    }
    enter_warp<true>(sh.map[buf], w, lane, r);
    IO *dx0 = static_cast<IO *>(p.dx) + (int64_t)t0 * p.D;
    float *dg0 = p.dg + (int64_t)t0 * p.D;
    const int n = l.any() ? tokens_of<TOK>(p, t0) : 0;
    // from the carry r: dx, dg and the carry of the token before; `past` is
    // h_{t-1}, less x_t for the complement
    auto write = [&](int i, float2 d, float2 ai, float2 past) {
      const float2 dt = add2(d, r);
      r = mul2(ai, dt);
      if (i < n && GDR_IN_BOUNDS((int64_t)t0 + i < p.tokens)) {
        store2<PAIRS>(dx0 + (int64_t)i * p.D, l, COMPLEMENT ? mul2(fresh<IO>(g_row(i), ai), dt) : dt);
        store2<PAIRS>(dg0 + (int64_t)i * p.D, l, mul2(r, past));
      }
    };
    auto less = [&](float2 y, float2 x) { return COMPLEMENT ? fma2(x, both(-1.f), y) : y; };
    if (!inside) {
      if (m.first) h = load_row<PAIRS>(p, p.initial_state, m.row_of(0), l);
      if (m.last) r = load_row<PAIRS>(p, p.dfinal, m.row_of(TOK - 1), l);
      float2 past[TOK];
#pragma unroll
      for (int i = 0; i < TOK; ++i) {
        const float2 x = x_of(i);
        past[i] = less(h, x);
        if (i < TOK - 1) h = advance(i, x, h);
      }
#pragma unroll
      for (int i = TOK - 1; i >= 0; --i) write(i, d_of(i), a[i], past[i]);
      if (m.first) store_state<PAIRS>(p, p.dinitial, m.row_of(0), l, r);
    } else {
      float2 past[TOK];  // (indexed by a running i: local memory)
#pragma unroll 2
      for (int i = 0; i < TOK; ++i) {
        if (m.first >> i & 1) h = load_row<PAIRS>(p, p.initial_state, m.row_of(i), l);
        past[i] = less(h, x_row(i));
        h = rolled(i, h);
      }
#pragma unroll 2
      for (int i = TOK - 1; i >= 0; --i) {
        if (m.last >> i & 1) r = load_row<PAIRS>(p, p.dfinal, m.row_of(i), l);
        write(i, d_row(i), decay<IO>(g_row(i)), past[i]);
        if (m.first >> i & 1) store_state<PAIRS>(p, p.dinitial, m.row_of(i), l, r);
      }
    }
    if (q.tile == 0) pass_empty(p, p.dfinal, p.dinitial, false, q.stripe * kWide, kWide);
    if (!more) return;
    if (!EARLY || inside) begin_copies(maps, rows, &sh.full[w], nq, w, lane);
    marked = next_marked;
    q = nq;
  }
}

// Before the scan kernels: zeroes the ticket and the chain's words, checks the
// packed offsets, writes the status word (once a call) and marks the tiles in which a
// sequence begins or ends.
__global__ void __launch_bounds__(256) glr_begin_kernel(GlrArgs p, int64_t words) {
  let_next_start();
  if (blockIdx.x == 0) {
    bool bad = false;
    if (p.cu_seqlens)
      for (int i = threadIdx.x; i <= p.num_seqs; i += blockDim.x) {
        const int32_t x = p.cu_seqlens[i];
        bad |= (i == 0 && x != 0) || (i == p.num_seqs && x != p.T) ||
               (i < p.num_seqs && p.cu_seqlens[i + 1] < x);
      }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
      if (bad) *p.status = KDA_DEVICE_BAD_CU_SEQLENS;
      else if (!p.keep_status) *p.status = KDA_DEVICE_OK;
      *p.ticket = (int32_t)p.first_ticket;
    }
  }
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = at; i < words / 2; i += step)  // (an even number, 16-byte aligned)
    reinterpret_cast<uint4 *>(p.tile_map)[i] = make_uint4(0, 0, 0, 0);
  if (p.cu_seqlens && p.num_seqs > 0)
    for (int64_t tile = at; tile < p.tiles; tile += step) {
      const int64_t t = tile * p.tile_tokens;
      int lo = 0, hi = p.num_seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_seqlens[mid] <= t) lo = mid;
        else hi = mid;
      }
      p.tile_marks[tile] = p.cu_seqlens[lo] == t || p.cu_seqlens[lo + 1] <= t + p.tile_tokens;
    }
}

// Without any token: what leaves each sequence is what enters it.
__global__ void __launch_bounds__(256) glr_no_tokens_kernel(GlrArgs p, bool backward) {
  if (failed(p)) return;
  const int n = blockIdx.x;
  const int64_t r = backward ? n : state_row(p, n);
  if (r < 0) return;
  const float *src = backward ? p.dfinal : p.initial_state;
  float *dst = backward ? p.dinitial : p.final_state;
  for (int c = threadIdx.x; c < p.D; c += blockDim.x) dst[r * p.D + c] = src ? src[r * p.D + c] : 0.f;
}

// One token for each sequence, the state in place: a thread a pair of channels, one
// pass.  16 x 2048 to 256 x 4096 bf16: 11 us a call, the host's time for it; in a
// replayed graph 1.5 and 5.4 us, 512 x 8192 14.2 = 4.7 TB/s (fp32 14.9 = 5.6).
template <typename IO, bool PAIRS, bool COMPLEMENT>
__global__ void __launch_bounds__(256) glr_step_kernel(GlrArgs p) {
  constexpr int V = PAIRS ? 2 : 1;
  const int c = (blockIdx.x * 256 + threadIdx.x) * V;
  if (c >= p.D) return;
  for (int n = blockIdx.y; n < p.num_seqs; n += gridDim.y) {
    const int64_t r = state_row(p, n);
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
    if (r >= 0 && GDR_IN_BOUNDS(r < p.num_slots && c + V <= p.D)) {
      const IO *x = static_cast<const IO *>(p.x) + n * p.ld_x + c;
      const float *g = p.g + n * p.ld_g + c;
      float *s = p.final_state + r * p.D + c;
      float xv[V], gv[V];
      if constexpr (PAIRS) {
        const float2 g2 = __ldg(reinterpret_cast<const float2 *>(g)), s2 = *reinterpret_cast<const float2 *>(s);
        gv[0] = g2.x; gv[1] = g2.y;
        h[0] = s2.x; h[1] = s2.y;
        if constexpr (sizeof(IO) == 2) {
          const uint32_t u = __ldg(reinterpret_cast<const unsigned int *>(x));
          xv[0] = bf16_lo(u); xv[1] = bf16_hi(u);
        } else {
          const float2 x2 = __ldg(reinterpret_cast<const float2 *>(x));
          xv[0] = x2.x; xv[1] = x2.y;
        }
      } else {
        gv[0] = __ldg(g);
        h[0] = *s;
        xv[0] = io<IO>::load(x);
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = fmaf(expf(gv[v]), h[v], COMPLEMENT ? -expm1f(gv[v]) * xv[v] : xv[v]);
      if constexpr (PAIRS) *reinterpret_cast<float2 *>(s) = make_float2(h[0], h[1]);
      else *s = h[0];
    }
    if (GDR_IN_BOUNDS(c + V <= p.D)) {
      IO *out = static_cast<IO *>(p.h) + (int64_t)n * p.D + c;
      if constexpr (!PAIRS) io<IO>::store(out, h[0]);
      else if constexpr (sizeof(IO) == 2) *reinterpret_cast<uint32_t *>(out) = pack_bf16x2(h[0], h[1]);
      else *reinterpret_cast<float2 *>(out) = make_float2(h[0], h[1]);
    }
  }
}

bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Two neighbouring channels a lane where the outputs' rows and the states allow it ...
bool pairs_ok(const GlrArgs &p) {
  const size_t e = p.bf16 ? 2 : 4;
  return p.D % 2 == 0 && p.ld_x % 2 == 0 && p.ld_g % 2 == 0 && p.ld_dh % 2 == 0 &&
         aligned_to(p.x, 2 * e) && aligned_to(p.h, 2 * e) && aligned_to(p.dh, 2 * e) &&
         aligned_to(p.dx, 2 * e) && aligned_to(p.g, 8) && aligned_to(p.dg, 8) &&
         aligned_to(p.initial_state, 8) && aligned_to(p.final_state, 8) &&
         aligned_to(p.dfinal, 8) && aligned_to(p.dinitial, 8) && aligned_to(p.chunk_states, 8);
}
// ... and the inputs' rows begin on 16 bytes, as tensor-map copies need.
bool maps_ok(const GlrArgs &p) {
  const int64_t v = p.bf16 ? 8 : 4;
  return pairs_ok(p) && p.ld_x % v == 0 && p.ld_dh % v == 0 && p.ld_g % 4 == 0 && aligned_to(p.x, 16) &&
         aligned_to(p.dh, 16) && aligned_to(p.g, 16);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Maps of a [tokens, D] tensor of type T for a warp's rows, zeros outside: N = 1,
// boxes of `tok` tokens x 64 channels; else every N-th row of each of the first N,
// from the 16-byte boundary at or before it, boxes of tok / N rows.
template <typename T, int N> bool make_maps(CUtensorMap (&m)[N], const void *base, const GlrArgs &p, int64_t ld, int tok) {
  auto fn = encode_fn();
  if (!fn) return false;
  for (int k = 0; k < N; ++k) {
    const bool there = k < p.tokens;  // (a row that is not is never looked at)
    const uintptr_t at = reinterpret_cast<uintptr_t>(base) + (there ? k * ld * sizeof(T) : 0);
    cuuint64_t dims[2] = {(cuuint64_t)p.D + at % 16 / sizeof(T), (cuuint64_t)(there ? (p.tokens - k + N - 1) / N : 1)};
    cuuint64_t strides[1] = {(cuuint64_t)ld * N * sizeof(T)};
    cuuint32_t box[2] = {kWide + (N > 1 ? N : 0), (cuuint32_t)(tok / N)}, estr[2] = {1, 1};
    if (fn(&m[k], sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
           reinterpret_cast<void *>(at / 16 * 16), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

cudaError_t launch_begin(const GlrArgs &p, cudaStream_t s) {
  const int64_t words = p.chained ? (p.tiles + p.groups) * p.pitch : 0;
  const int64_t most = words > p.tiles ? words : p.tiles, want = (most + 2047) / 2048, cap = 4 * sm_count();
  TraceScope tr("glr_begin_kernel", s);
  glr_begin_kernel<<<(unsigned)(want < 1 ? 1 : want > cap ? cap : want), 256, 0, s>>>(p, words);
  return cudaGetLastError();
}

cudaError_t launch_no_tokens(const GlrArgs &p, bool backward, cudaStream_t s) {
  if (p.num_seqs == 0 || !(backward ? p.dinitial : p.final_state)) return cudaSuccess;
  TraceScope tr("glr_no_tokens_kernel", s);
  glr_no_tokens_kernel<<<p.num_seqs, 256, 0, s>>>(p, backward);
  return cudaGetLastError();
}

// The tiles of a launch with TOK tokens a warp, and whether they wait for one
// another: not where each begins with a sequence's first token.
template <int TOK> GlrArgs with_tiles(const GlrArgs &a) {
  GlrArgs p = a;
  p.tile_tokens = kWarps * TOK;
  p.tiles = (p.tokens + p.tile_tokens - 1) / p.tile_tokens;
  p.stripes = (p.D + kWide - 1) / kWide;
  p.chained = p.tiles > 1 && (p.cu_seqlens || p.T > p.tile_tokens || p.tile_tokens % p.T != 0);
  p.groups = (p.tiles + Chain<TOK>::kGroup - 1) / Chain<TOK>::kGroup;
  p.carry = p.tile_map + p.tiles * p.pitch;
  return p;
}

// Blocks of a scan kernel that run at once on the current device (asked once a device).
template <typename K> cudaError_t resident_blocks(K kernel, std::atomic<int> *cache, size_t smem, int *blocks) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool keep = dev >= 0 && dev < kCachedDevices;
  *blocks = keep ? cache[dev].load(std::memory_order_relaxed) : 0;
  if (*blocks > 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  int per_sm = 0;
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem);
  if (e != cudaSuccess) return e;
  *blocks = sm_count() * (per_sm > 0 ? per_sm : 1);
  if (keep) cache[dev].store(*blocks, std::memory_order_relaxed);
  return cudaSuccess;
}

// Launches a scan kernel with as many blocks as run at once, or one a tile.
template <auto KERNEL, typename MAPS>
cudaError_t launch_tiles(const char *name, size_t smem, const GlrArgs &p, const MAPS &maps, cudaStream_t s) {
  static std::atomic<int> cache[kCachedDevices];
  int most = 0;
  cudaError_t e = resident_blocks(KERNEL, cache, smem, &most);
  if (e != cudaSuccess) return e;
  const int64_t tiles = p.tiles * p.stripes;
  TraceScope tr(name, s);
  return launch_behind(KERNEL, dim3((unsigned)(tiles < most ? tiles : most)), dim3(kThreads), smem, s, p, maps);
}

template <typename IO, bool PAIRS, bool COMPLEMENT, bool STATES_ONLY>
cudaError_t launch_scan(const GlrArgs &a, cudaStream_t s) {
  constexpr int TOK = FwdShape<IO, PAIRS, COMPLEMENT>::kTok;
  const GlrArgs p = with_tiles<TOK>(a);
  cudaError_t e = launch_begin(p, s);
  if (e != cudaSuccess) return e;
  if (p.tiles == 0) return launch_no_tokens(p, false, s);
  GlrMaps<IO, PAIRS, false> maps{};
  if (!(make_maps<IO>(maps.x, p.x, p, p.ld_x, TOK) && make_maps<float>(maps.g, p.g, p, p.ld_g, TOK)))
    return cudaErrorInvalidValue;
  return launch_tiles<glr_scan_kernel<IO, PAIRS, COMPLEMENT, STATES_ONLY>>(
      "glr_scan_kernel", kWarps * sizeof(WarpRows<IO, PAIRS, TOK, false>), p, maps, s);
}

template <typename IO, bool PAIRS, bool COMPLEMENT>
cudaError_t launch_fwd(const GlrArgs &a, cudaStream_t s) {
  return launch_scan<IO, PAIRS, COMPLEMENT, false>(a, s);
}

template <typename IO, bool PAIRS, bool COMPLEMENT>
cudaError_t launch_bwd(const GlrArgs &a, cudaStream_t s) {
  constexpr int TOK = BwdShape<IO, COMPLEMENT>::kTok;
  GlrArgs p = with_tiles<TOK>(a);
  p.first_ticket = 0;
  cudaError_t e = cudaSuccess;
  if (p.own_chunks && p.tiles > 0) {
    e = launch_scan<IO, PAIRS, COMPLEMENT, true>(a, s);
    p.keep_status = true;
  }
  if (e == cudaSuccess) e = launch_begin(p, s);
  if (e != cudaSuccess) return e;
  if (p.tiles == 0) return launch_no_tokens(p, true, s);
  GlrMaps<IO, PAIRS, true> maps{};
  if (!(make_maps<IO>(maps.x, p.x, p, p.ld_x, TOK) && make_maps<float>(maps.g, p.g, p, p.ld_g, TOK) &&
        make_maps<IO>(maps.dh, p.dh, p, p.ld_dh, TOK)))
    return cudaErrorInvalidValue;
  return launch_tiles<glr_gradient_kernel<IO, PAIRS, COMPLEMENT>>(
      "glr_gradient_kernel", kWarps * sizeof(WarpRows<IO, PAIRS, TOK, true>), p, maps, s);
}

template <typename IO, bool PAIRS, bool COMPLEMENT>
cudaError_t launch_step(const GlrArgs &p, cudaStream_t s) {
  TraceScope tr("glr_step_kernel", s);
  const int wide = PAIRS ? 512 : 256;
  const dim3 grid((unsigned)((p.D + wide - 1) / wide), (unsigned)(p.num_seqs < 65535 ? p.num_seqs : 65535));
  glr_step_kernel<IO, PAIRS, COMPLEMENT><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

#define GDR_GLR_DISPATCH(fn, pairs)                                                      \
  do {                                                                                   \
    const bool two = pairs;                                                              \
    if (p.bf16)                                                                          \
      return p.complement ? (two ? fn<__nv_bfloat16, true, true>(p, s) : fn<__nv_bfloat16, false, true>(p, s))   \
                          : (two ? fn<__nv_bfloat16, true, false>(p, s) : fn<__nv_bfloat16, false, false>(p, s)); \
    return p.complement ? (two ? fn<float, true, true>(p, s) : fn<float, false, true>(p, s))   \
                        : (two ? fn<float, true, false>(p, s) : fn<float, false, false>(p, s)); \
  } while (0)

}  // namespace

GDR_DEFINE_OOB_COUNTER(oob_count_glr)

cudaError_t launch_glr_fwd(const GlrArgs &p, cudaStream_t s) { GDR_GLR_DISPATCH(launch_fwd, maps_ok(p)); }
cudaError_t launch_glr_bwd(const GlrArgs &p, cudaStream_t s) { GDR_GLR_DISPATCH(launch_bwd, maps_ok(p)); }
cudaError_t launch_glr_step(const GlrArgs &p, cudaStream_t s) { GDR_GLR_DISPATCH(launch_step, pairs_ok(p)); }

}  // namespace gdr
