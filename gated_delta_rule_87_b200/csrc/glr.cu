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
// (A, H) with out = A in + H.  The decay product of a span is exp of the sum
// of its g, so a long memory loses no precision to the rounding of each a_t.
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
// it (and for tensor-map copies); else 32 apart, any alignment.
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

// Two channels of one token as they are stored.
template <typename IO> struct Raw;
template <> struct Raw<float> {
  float r[2];
  __device__ __forceinline__ float at(int v) const { return r[v]; }
};
template <> struct Raw<__nv_bfloat16> {
  uint32_t r;
  __device__ __forceinline__ float at(int v) const { return v ? bf16_hi(r) : bf16_lo(r); }
};

// Shared memory: a lane's two channels of a row.
template <bool PAIRS> __device__ __forceinline__ Raw<float> read_row(const float *row, int lane) {
  Raw<float> x;
  if constexpr (PAIRS) {
    const float2 v = reinterpret_cast<const float2 *>(row)[lane];
    x.r[0] = v.x; x.r[1] = v.y;
  } else {
    x.r[0] = row[lane]; x.r[1] = row[lane + 32];
  }
  return x;
}
template <bool PAIRS> __device__ __forceinline__ Raw<__nv_bfloat16> read_row(const __nv_bfloat16 *row, int lane) {
  Raw<__nv_bfloat16> x;
  if constexpr (PAIRS) {
    x.r = reinterpret_cast<const uint32_t *>(row)[lane];
  } else {
    const unsigned short *h = reinterpret_cast<const unsigned short *>(row);
    x.r = (uint32_t)h[lane] | (uint32_t)h[lane + 32] << 16;
  }
  return x;
}

template <bool PAIRS> __device__ __forceinline__ void write_row(float *row, int lane, const float (&x)[2]) {
  if constexpr (PAIRS) {
    reinterpret_cast<float2 *>(row)[lane] = make_float2(x[0], x[1]);
  } else {
    row[lane] = x[0]; row[lane + 32] = x[1];
  }
}

// Global memory: plain (coherent) accesses, states are updated in place by some calls.
template <bool PAIRS> __device__ __forceinline__ void load2(const float *p, const Lane<PAIRS> &l, float (&x)[2]) {
  if constexpr (PAIRS) {
    const float2 v = *reinterpret_cast<const float2 *>(p + l.c);
    x[0] = v.x; x[1] = v.y;
  } else {
    x[0] = p[l.c];
    x[1] = l.on[1] ? p[l.c + 32] : 0.f;
  }
}
template <bool PAIRS, typename IO> __device__ __forceinline__ void store2(IO *p, const Lane<PAIRS> &l, const float (&x)[2]) {
  if constexpr (!PAIRS) {
    io<IO>::store(p + l.c, x[0]);
    if (l.on[1]) io<IO>::store(p + l.c + 32, x[1]);
  } else if constexpr (sizeof(IO) == 4) {
    *reinterpret_cast<float2 *>(p + l.c) = make_float2(x[0], x[1]);
  } else {
    *reinterpret_cast<uint32_t *>(p + l.c) = pack_bf16x2(x[0], x[1]);
  }
}

// The decay of one token.  With bf16 activations the fast exponential: its error
// (2^-22 of the value) enters the state of a span of at most 16 tokens only,
// the decay of longer spans comes from the sum of their g.
template <typename IO> __device__ __forceinline__ float decay(float g) {
  if constexpr (sizeof(IO) == 2) {
    float a;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(g * 1.44269504f));  // log2 e
    return a;
  } else {
    return expf(g);
  }
}
// 1 - a of one token: near 0 the series of -expm1(g), whose first term left out
// is below 2^-22 of the value (bf16 activations) or 2^-28, else the difference,
// which then loses less than two bits.
template <typename IO> __device__ __forceinline__ float fresh(float g, float a) {
  float s = 1.f / 5040.f;
  if constexpr (sizeof(IO) == 4) {
    s = 1.f / 362880.f;
    s = fmaf(s, g, 1.f / 40320.f);
    s = fmaf(s, g, 1.f / 5040.f);
  }
  s = fmaf(s, g, 1.f / 720.f);
  s = fmaf(s, g, 1.f / 120.f);
  s = fmaf(s, g, 1.f / 24.f);
  s = fmaf(s, g, 1.f / 6.f);
  s = fmaf(s, g, 0.5f);
  s = fmaf(s, g, 1.f);
  return g > -0.5f ? -g * s : 1.f - a;
}

// Which of a warp's TOK tokens begin or end a sequence (bit i: token t0 + i), and,
// in lane i, the sequence of token t0 + i.
struct Marks {
  uint32_t first, last;
  int seq;
};
template <int TOK> __device__ __forceinline__ Marks find_marks(const GlrArgs &p, uint32_t t0, int lane) {
  static_assert(TOK <= 32, "a lane a token");
  Marks m;
  bool f = false, l = false;
  m.seq = 0;
  const uint32_t t = t0 + lane;
  if (lane < TOK && t < (uint32_t)p.tokens) {
    if (p.cu_seqlens) {  // the last sequence that starts at or before t (empty ones start there too)
      int lo = 0, hi = p.num_seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((uint32_t)__ldg(p.cu_seqlens + mid) <= t) lo = mid;
        else hi = mid;
      }
      m.seq = lo;
      f = (uint32_t)__ldg(p.cu_seqlens + lo) == t;
      l = (uint32_t)__ldg(p.cu_seqlens + lo + 1) == t + 1;
    } else {
      m.seq = (int)(t / (uint32_t)p.T);
      const uint32_t r = t - (uint32_t)m.seq * (uint32_t)p.T;
      f = r == 0;
      l = r == (uint32_t)p.T - 1;
    }
  }
  m.first = __ballot_sync(0xffffffffu, f);
  m.last = __ballot_sync(0xffffffffu, l);
  return m;
}

// Row of sequence n's state in the states or the pool, or -1 (no slot).
__device__ __forceinline__ int64_t state_row(const GlrArgs &p, int n) {
  if (!p.state_slots) return n;
  const int64_t s = __ldg(p.state_slots + n);
  return s >= 0 && s < p.num_slots ? s : -1;
}

// The initial state of sequence n.
template <bool PAIRS>
__device__ __forceinline__ void initial_of(const GlrArgs &p, int n, const Lane<PAIRS> &l, float (&h0)[2]) {
  h0[0] = h0[1] = 0.f;
  if (!p.initial_state) return;
  const int64_t r = state_row(p, n);
  if (l.any() && r >= 0 && GDR_IN_BOUNDS(n < p.num_seqs && r < p.num_slots))
    load2<PAIRS>(p.initial_state + r * p.D, l, h0);
}

__device__ __forceinline__ bool bad_offsets(const GlrArgs &p) {
  return p.cu_seqlens && *reinterpret_cast<const volatile int32_t *>(p.status) != KDA_DEVICE_OK;
}

// ---- maps of spans ------------------------------------------------------
// A span of tokens takes what enters it, `in`, to A in + H, or to H where it is
// closed.  A >= 0 is kept with its sign turned, a closed span as +1 in its place.
// All channels of a span are closed or none.
struct Map2 {  // of a lane's two channels
  float A[2], H[2];
};
constexpr float kClosed = 1.f;
__device__ __forceinline__ float through(float A, float H, float in) { return A > 0.f ? H : fmaf(-A, in, H); }
__device__ __forceinline__ void through(const Map2 &m, float (&x)[2]) {
  x[0] = through(m.A[0], m.H[0], x[0]);
  x[1] = through(m.A[1], m.H[1], x[1]);
}
// The map of n spans one after the other (n known where it is unrolled).
template <int N> __device__ __forceinline__ Map2 joined(const Map2 (&t)[N]) {
  Map2 m = t[0];
  bool closed = false;
#pragma unroll
  for (int j = 0; j < N; ++j) closed |= t[j].A[0] > 0.f;
  if (!closed) {
#pragma unroll
    for (int j = 1; j < N; ++j)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        m.H[v] = fmaf(-t[j].A[v], m.H[v], t[j].H[v]);
        m.A[v] = -(m.A[v] * t[j].A[v]);
      }
  } else {
#pragma unroll
    for (int j = 1; j < N; ++j) through(t[j], m.H);
    m.A[0] = m.A[1] = kClosed;
  }
  return m;
}

struct TileShared {
  // the warps' maps; a tile's are read until its end, while the next one's are written
  Map2 map[2][kWarps][32];
  Map2 before[kWarps][32];  // of earlier tiles, a part a warp
  uint64_t full[kWarps];    // a warp's copies have landed
  uint32_t step;            // of the block's next tile
  int stripe;
};

// ---- the chain of tiles -------------------------------------------------
// Blocks take tiles in order of a ticket, each its own in rising order, so
// every tile that another waits for is done or in the hands of a block that
// waits for earlier ones only: the lowest open ticket always proceeds.  In
// groups of kGroup tiles a tile publishes its map as soon as it has it; what
// enters a tile is what enters its group, through the maps of the group's tiles
// before it; the last tile of a group publishes what leaves the group.  Which
// values are joined, and in which order, depends on the sizes alone, never on
// timing.
//
// A channel's map goes through the workspace as one 64-bit word (A above, H
// below), which is its own flag: 0 is not there yet, and A is never +0.  So a
// hand-over is one store and one polling load, without a fence.  The rows of
// words are as wide as the tiles (`pitch`), so every lane has its own.
constexpr int kGroup = 16, kPart = kGroup / kWarps;
static_assert(kGroup >= kGlrShortestGroup, "the workspace counts groups of at least this length");
constexpr uint32_t kMaxChainPolls = 1u << 20;  // about a second

struct Words {
  uint64_t u[2];
  __device__ __forceinline__ bool here() const { return min((uint32_t)(u[0] >> 32), (uint32_t)(u[1] >> 32)) != 0; }
  __device__ __forceinline__ Map2 map() const {
    Map2 m;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      m.A[v] = __uint_as_float((uint32_t)(u[v] >> 32));
      m.H[v] = __uint_as_float((uint32_t)u[v]);
    }
    return m;
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
template <bool PAIRS> __device__ __forceinline__ void store_words(uint64_t *p, const Map2 &m) {
  uint64_t u[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) u[v] = (uint64_t)__float_as_uint(m.A[v]) << 32 | __float_as_uint(m.H[v]);
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
  __device__ __forceinline__ int in_group() const { return step % kGroup; }
  __device__ __forceinline__ uint32_t group() const { return step / kGroup; }
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
  if (poll < kMaxChainPolls) return false;
  *p.status = KDA_DEVICE_TIMEOUT;
  return true;
}

// After the warps have shared their maps, one of them publishes the tile's,
// unless the tile ends its group.
template <bool PAIRS, bool REV>
__device__ __forceinline__ void publish_tile(const GlrArgs &p, const TileShared &sh, int buf, const Place &q,
                                             int c, int lane) {
  Map2 t[kWarps];
#pragma unroll
  for (int k = 0; k < kWarps; ++k) t[k] = sh.map[buf][REV ? kWarps - 1 - k : k][lane];
  if (GDR_IN_BOUNDS(q.step < p.tiles && c < p.pitch))
    store_words<PAIRS>(p.tile_map + (int64_t)q.step * p.pitch + c, joined(t));
}

// What enters the tile.  Each warp joins its part of the group's earlier maps,
// then all wait for what enters the group and take it through the parts.  That
// wait is the serial part of the chain: the tile that ends a group sends on
// what leaves it at once.  Every thread of the block takes part.  False: a wait
// gave up.
template <bool PAIRS, bool REV>
__device__ __forceinline__ bool enter_tile(const GlrArgs &p, TileShared &sh, int buf, const Place &q, int c, int w,
                                           int lane, float (&in)[2]) {
  const int at = q.in_group(), n = at - w * kPart;  // maps to join (at most kPart)
  bool ok = true;
  // (the carry of a group begun long ago is there by now, or looked at again below)
  const bool behind = q.step >= kGroup && GDR_IN_BOUNDS(q.group() <= p.groups && c < p.pitch);
  const uint64_t *carry = p.carry + ((int64_t)q.group() - 1) * p.pitch + c;
  Words u;
  u.u[0] = u.u[1] = 0;
  if (behind) load_words<PAIRS>(carry, u);
  if (n > 0 && GDR_IN_BOUNDS(q.step < p.tiles && c < p.pitch)) {
    const uint64_t *from = p.tile_map + (int64_t)(q.step - n) * p.pitch + c;
    Words t[kPart];
#pragma unroll
    for (int j = 0; j < kPart; ++j) {
      t[j].u[0] = t[j].u[1] = (uint64_t)__float_as_uint(-1.f) << 32;  // nothing changes
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
#pragma unroll
    for (int j = 0; j < kPart; ++j) m[j] = t[j].map();
    sh.before[w][lane] = joined(m);
  }
  if (__syncthreads_or(!ok)) return false;
  Map2 part[kWarps];
  bool closed = false;  // nothing to wait for where a sequence began since
#pragma unroll
  for (int k = 0; k < kWarps; ++k)
    if (k * kPart < at) {
      part[k] = sh.before[k][lane];
      closed |= part[k].A[0] > 0.f;
    }
  in[0] = in[1] = 0.f;
  if (behind && !closed) {
    for (uint32_t poll = 0; !__all_sync(0xffffffffu, u.here()); ++poll) {
      if (give_up(p, poll)) {
        ok = false;  // the block finds out at its next barrier
        break;
      }
      load_words<PAIRS>(carry, u);
    }
    const Map2 m = u.map();
    in[0] = m.H[0];
    in[1] = m.H[1];
  }
#pragma unroll
  for (int k = 0; k < kWarps; ++k)
    if (k * kPart < at) through(part[k], in);
  if (ok && at == kGroup - 1 && w == (REV ? 0 : kWarps - 1) && GDR_IN_BOUNDS(q.group() < p.groups && c < p.pitch)) {
    Map2 out;
    out.H[0] = in[0];
    out.H[1] = in[1];
#pragma unroll
    for (int k = 0; k < kWarps; ++k) through(sh.map[buf][REV ? kWarps - 1 - k : k][lane], out.H);
    out.A[0] = out.A[1] = kClosed;
    store_words<PAIRS>(p.carry + (int64_t)q.group() * p.pitch + c, out);
  }
  return ok;
}

// `x`, what enters the tile, becomes what enters warp w.
template <bool REV>
__device__ __forceinline__ void enter_warp(const Map2 (&map)[kWarps][32], int w, int lane, float (&x)[2]) {
#pragma unroll
  for (int k = 0; k < kWarps - 1; ++k) {
    const int j = REV ? kWarps - 1 - k : k;
    if (REV ? j > w : j < w) through(map[j][lane], x);
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
// the path without marks).
__device__ __forceinline__ bool has_marks(const GlrArgs &p, uint32_t tile) {
  if (p.cu_seqlens) return __ldg(p.tile_marks + tile) != 0;
  const uint32_t t = tile * p.tile_tokens, r = t % (uint32_t)p.T;
  return r == 0 || r + p.tile_tokens >= (uint32_t)p.T;
}

// ---- the kernels --------------------------------------------------------
// Persistent blocks of four warps; a tile is TOK tokens a warp and 64 channels.
// Each warp copies its own rows to shared memory (a tensor-map copy a tensor, or
// lane by lane where rows are not aligned) and waits for them alone.  In the
// first pass over a tile its rows go to registers, so that the next tile's
// copies run while this one waits for what enters it and is written: one read
// of each input.  What an SM moves is what its blocks hold (registers and the
// copies under way) over the time a tile takes, two or three L2 round trips.
//
// A tile in which a sequence begins or ends takes rolled loops instead, over the
// rows in shared memory, and its block's next copies begin after it.
template <typename IO, int TOK> struct WarpRows {
  float g[TOK][kWide];
  IO x[TOK][kWide];
};
template <typename IO, int TOK> struct WarpRowsBwd : WarpRows<IO, TOK> {
  IO dh[TOK][kWide];
};
struct GlrMaps {
  CUtensorMap x, g, dh;
};

// Tokens of a warp that exist.
template <int TOK> __device__ __forceinline__ int tokens_of(const GlrArgs &p, uint32_t t0) {
  const int64_t left = p.tokens - (int64_t)t0;
  return left <= 0 ? 0 : left < TOK ? (int)left : TOK;
}

// Lane copies of one tensor's rows; zeros where nothing is.
template <typename IO, int TOK>
__device__ __forceinline__ void copy_rows(const GlrArgs &p, IO (&to)[TOK][kWide], const void *from, int64_t ld,
                                          uint32_t t0, const Lane<false> &l, int lane) {
  const IO *src = static_cast<const IO *>(from);
  const int n = tokens_of<TOK>(p, t0);
  int64_t off = (int64_t)t0 * ld + l.c;
  if constexpr (sizeof(IO) == 4) {
#pragma unroll
    for (int i = 0; i < TOK; ++i, off += ld)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const bool ok = i < n && l.on[v] && GDR_IN_BOUNDS((int64_t)t0 + i < p.tokens && l.c + 32 * v < p.D);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(&to[i][lane + 32 * v])),
                     "l"(ok ? src + off + 32 * v : src), "r"(ok ? 4 : 0) : "memory");
      }
  } else {  // a single bf16 is too short for an asynchronous copy
    IO t[TOK][2];
#pragma unroll
    for (int i = 0; i < TOK; ++i, off += ld)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const bool ok = i < n && l.on[v] && GDR_IN_BOUNDS((int64_t)t0 + i < p.tokens && l.c + 32 * v < p.D);
        t[i][v] = ok ? __ldg(src + off + 32 * v) : __float2bfloat16_rn(0.f);
      }
#pragma unroll
    for (int i = 0; i < TOK; ++i)
#pragma unroll
      for (int v = 0; v < 2; ++v) to[i][lane + 32 * v] = t[i][v];
  }
}

// Begins the copies of a warp's rows of a tile.
template <typename IO, bool PAIRS, bool BWD, int TOK, typename ROWS>
__device__ __forceinline__ void begin_copies(const GlrArgs &p, const GlrMaps &maps, ROWS &rows, uint64_t *full,
                                             const Place &q, int w, int lane) {
  const uint32_t t0 = q.tile * (kWarps * TOK) + w * TOK;
  if constexpr (PAIRS) {
    __syncwarp();  // the rows have been read by every lane
    if (lane == 0) {
      const int c0 = q.stripe * kWide;
      tc::mbar_arrive_expect_tx(full, sizeof(ROWS));
      tc::tma_load_2d(rows.g, &maps.g, c0, (int)t0, full);
      tc::tma_load_2d(rows.x, &maps.x, c0, (int)t0, full);
      if constexpr (BWD) tc::tma_load_2d(rows.dh, &maps.dh, c0, (int)t0, full);
    }
  } else {
    const Lane<false> l(q.stripe, p.D);
    copy_rows<float, TOK>(p, rows.g, p.g, p.ld_g, t0, l, lane);
    copy_rows<IO, TOK>(p, rows.x, p.x, p.ld_x, t0, l, lane);
    if constexpr (BWD) copy_rows<IO, TOK>(p, rows.dh, p.dh, p.ld_dh, t0, l, lane);
  }
}
template <bool PAIRS>
__device__ __forceinline__ bool copies_done(const GlrArgs &p, uint64_t *full, uint32_t parity) {
  if constexpr (PAIRS) return tc::mbar_wait_warp(full, parity, p.status, KDA_DEVICE_TIMEOUT);
  asm volatile("cp.async.wait_all;" ::: "memory");
  return true;
}
__device__ __forceinline__ void init_barriers(TileShared &sh) {
  if (threadIdx.x < kWarps) tc::mbar_init(&sh.full[threadIdx.x], 1);
  tc::mbar_fence_init();
}

// Tokens a warp, and blocks an SM by their registers.  The chain and the barriers
// cost about as much for a long tile as for a short one, so a tile is as long as
// the registers allow: forward in bf16, 32 tokens a warp (a and the packed x in
// 96 registers, three blocks) against 16 (four blocks).
template <typename IO, bool PAIRS, bool COMPLEMENT> struct FwdShape {
  static constexpr bool kLong = PAIRS && sizeof(IO) == 2 && !COMPLEMENT;
  static constexpr int kTok = kLong ? 32 : 16, kBlocks = kLong ? 3 : 4;
};
// Backward: in bf16 x and dh go to registers as well; else (x and dh too wide, or
// g needed again) they are read from shared memory in both passes, and the next
// copies begin after the second.
template <typename IO, bool COMPLEMENT> struct BwdShape {
  static constexpr bool kEarly = sizeof(IO) == 2 && !COMPLEMENT;
  static constexpr int kTok = 16, kBlocks = kEarly ? 3 : 4;
};

// Forward.  STATES_ONLY: only the saved chunk states are written.
template <typename IO, bool PAIRS, bool COMPLEMENT, bool STATES_ONLY>
__global__ void __launch_bounds__(kThreads, (FwdShape<IO, PAIRS, COMPLEMENT>::kBlocks))
glr_scan_kernel(const __grid_constant__ GlrArgs p, const __grid_constant__ GlrMaps maps) {
  constexpr int TOK = FwdShape<IO, PAIRS, COMPLEMENT>::kTok;
  __shared__ TileShared sh;
  extern __shared__ __align__(128) unsigned char tile_bytes[];
  if (bad_offsets(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  auto &rows = reinterpret_cast<WarpRows<IO, TOK> *>(tile_bytes)[w];
  uint32_t ticket = 0, parity = 0;
  init_barriers(sh);
  if (threadIdx.x == 0) ticket = next_ticket(p, sh, blockIdx.x - gridDim.x);
  __syncthreads();
  Place q = taken<false>(p, sh);
  if (q.step >= p.tiles) return;
  __syncthreads();
  begin_copies<IO, PAIRS, false, TOK>(p, maps, rows, &sh.full[w], q, w, lane);
  bool marked = has_marks(p, q.tile), alive = true;
  while (true) {
    if (threadIdx.x == 0) ticket = next_ticket(p, sh, ticket);
    Lane<PAIRS> l(q.stripe, p.D);
    const uint32_t t0 = q.tile * (kWarps * TOK) + w * TOK;
    Marks m;
    m.first = m.last = 0;
    m.seq = 0;
    if (marked) m = find_marks<TOK>(p, t0, lane);
    alive &= copies_done<PAIRS>(p, &sh.full[w], parity);
    const int buf = parity;
    parity ^= 1;
    // the map of the warp's tokens; b of a token is x, or (1 - a) x
    float a[TOK][2], b[COMPLEMENT ? TOK : 1][2], gs[2] = {0.f, 0.f}, h[2] = {0.f, 0.f};
    Raw<IO> x[COMPLEMENT ? 1 : TOK];
    auto b_of = [&](int i, int v) { return COMPLEMENT ? b[COMPLEMENT ? i : 0][v] : x[COMPLEMENT ? 0 : i].at(v); };
    auto rolled = [&](int i) {  // the state h after token i, from shared memory
      const Raw<float> g = read_row<PAIRS>(rows.g[i], lane);
      const Raw<IO> xi = read_row<PAIRS>(rows.x[i], lane);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float ai = decay<IO>(g.at(v));
        h[v] = fmaf(ai, h[v], COMPLEMENT ? fresh<IO>(g.at(v), ai) * xi.at(v) : xi.at(v));
        gs[v] += g.at(v);
      }
    };
    if (!marked) {
#pragma unroll
      for (int i = 0; i < TOK; ++i) {
        const Raw<float> g = read_row<PAIRS>(rows.g[i], lane);
        const Raw<IO> xi = read_row<PAIRS>(rows.x[i], lane);
        if (!COMPLEMENT) x[COMPLEMENT ? 0 : i] = xi;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          a[i][v] = decay<IO>(g.at(v));
          if (COMPLEMENT) b[COMPLEMENT ? i : 0][v] = fresh<IO>(g.at(v), a[i][v]) * xi.at(v);
          gs[v] += g.at(v);
        }
      }
#pragma unroll
      for (int i = 0; i < TOK; ++i)
#pragma unroll
        for (int v = 0; v < 2; ++v) h[v] = fmaf(a[i][v], h[v], b_of(i, v));
    } else {
      // The state after a start takes the place of its g: the initial state is
      // read once, before the map is published (the sequence's last tile may
      // write the final state over it as soon as that is done).
      for (int i = 0; i < TOK; ++i) {
        const bool start = m.first >> i & 1;
        if (start) initial_of<PAIRS>(p, __shfl_sync(0xffffffffu, m.seq, i), l, h);
        rolled(i);
        if (start) write_row<PAIRS>(rows.g[i], lane, h);
      }
    }
    sh.map[buf][w][lane] = {{m.first ? kClosed : -expf(gs[0]), m.first ? kClosed : -expf(gs[1])}, {h[0], h[1]}};
    if (__syncthreads_or(!alive)) return;  // a wait gave up; no copy is under way
    if (p.chained && w == kWarps - 1 && q.in_group() != kGroup - 1) publish_tile<PAIRS, false>(p, sh, buf, q, l.c, lane);
    const Place nq = taken<false>(p, sh);
    const bool more = nq.step < p.tiles;
    if (more && !marked) begin_copies<IO, PAIRS, false, TOK>(p, maps, rows, &sh.full[w], nq, w, lane);
    const bool next_marked = more && has_marks(p, nq.tile);
    h[0] = h[1] = 0.f;
    if (p.chained) {
      alive = enter_tile<PAIRS, false>(p, sh, buf, q, l.c, w, lane, h);
      if (!alive) l.on[0] = l.on[1] = false;  // writes nothing, and ends at the next barrier
    } else {
      __syncthreads();  // the next ticket is read before it is replaced
    }
    enter_warp<false>(sh.map[buf], w, lane, h);
    // (a chunk of 64 tokens begins with every warp of 64, 32 or 16 tokens that divides it)
    if (p.chunk_states && t0 % kGlrChunk == 0 && l.any() && t0 < p.tokens && GDR_IN_BOUNDS(t0 / kGlrChunk < p.chunks))
      store2<PAIRS>(p.chunk_states + (int64_t)(t0 / kGlrChunk) * p.D, l, h);
    if (!STATES_ONLY) {
      IO *out = static_cast<IO *>(p.h) + (int64_t)t0 * p.D;
      const int n = l.any() ? tokens_of<TOK>(p, t0) : 0;
      if (!marked) {
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
#pragma unroll
          for (int v = 0; v < 2; ++v) h[v] = fmaf(a[i][v], h[v], b_of(i, v));
          if (i < n && GDR_IN_BOUNDS((int64_t)t0 + i < p.tokens)) store2<PAIRS>(out + (int64_t)i * p.D, l, h);
        }
      } else {
        for (int i = 0; i < TOK; ++i) {
          if (m.first >> i & 1) {
            const Raw<float> g = read_row<PAIRS>(rows.g[i], lane);
            h[0] = g.at(0);
            h[1] = g.at(1);
          } else {
            rolled(i);
          }
          if (i < n && GDR_IN_BOUNDS((int64_t)t0 + i < p.tokens)) store2<PAIRS>(out + (int64_t)i * p.D, l, h);
          const int s = __shfl_sync(0xffffffffu, m.seq, i);
          if ((m.last >> i & 1) && p.final_state) {
            const int64_t r = state_row(p, s);
            if (l.any() && r >= 0 && GDR_IN_BOUNDS(s < p.num_seqs && r < p.num_slots))
              store2<PAIRS>(p.final_state + r * p.D, l, h);
          }
        }
      }
      if (q.tile == 0) pass_empty(p, p.initial_state, p.final_state, true, q.stripe * kWide, kWide);
    }
    if (!more) return;
    if (marked) begin_copies<IO, PAIRS, false, TOK>(p, maps, rows, &sh.full[w], nq, w, lane);
    marked = next_marked;
    q = nq;
  }
}

// Backward: the states again from what enters the tile (saved), the gradients
// from what enters it from the tokens after it (chained).
template <typename IO, bool PAIRS, bool COMPLEMENT>
__global__ void __launch_bounds__(kThreads, (BwdShape<IO, COMPLEMENT>::kBlocks))
glr_gradient_kernel(const __grid_constant__ GlrArgs p, const __grid_constant__ GlrMaps maps) {
  constexpr bool EARLY = BwdShape<IO, COMPLEMENT>::kEarly;
  constexpr int TOK = BwdShape<IO, COMPLEMENT>::kTok;
  static_assert(kWarps * TOK == kGlrChunk, "a tile is a chunk: its saved state enters it");
  __shared__ TileShared sh;
  __shared__ Map2 states[kWarps][32];  // the warps' maps of the states
  extern __shared__ __align__(128) unsigned char tile_bytes[];
  if (bad_offsets(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  auto &rows = reinterpret_cast<WarpRowsBwd<IO, TOK> *>(tile_bytes)[w];
  uint32_t ticket = 0, parity = 0;
  init_barriers(sh);
  if (threadIdx.x == 0) ticket = next_ticket(p, sh, blockIdx.x - gridDim.x);
  __syncthreads();
  Place q = taken<true>(p, sh);
  if (q.step >= p.tiles) return;
  __syncthreads();
  begin_copies<IO, PAIRS, true, TOK>(p, maps, rows, &sh.full[w], q, w, lane);
  bool marked = has_marks(p, q.tile), alive = true;
  while (true) {
    if (threadIdx.x == 0) ticket = next_ticket(p, sh, ticket);
    Lane<PAIRS> l(q.stripe, p.D);
    const uint32_t t0 = q.tile * (kWarps * TOK) + w * TOK;
    float h[2] = {0.f, 0.f}, s[2] = {0.f, 0.f}, r[2] = {0.f, 0.f}, gs[2] = {0.f, 0.f};
    if (l.any() && GDR_IN_BOUNDS(q.tile < p.chunks)) load2<PAIRS>(p.chunk_states + (int64_t)q.tile * p.D, l, h);
    Marks m;
    m.first = m.last = 0;
    m.seq = 0;
    if (marked) m = find_marks<TOK>(p, t0, lane);
    alive &= copies_done<PAIRS>(p, &sh.full[w], parity);
    const int buf = parity;
    parity ^= 1;
    float a[TOK][2];
    Raw<IO> xk[EARLY ? TOK : 1], dk[EARLY ? TOK : 1];
    auto x_of = [&](int i) { return EARLY ? xk[EARLY ? i : 0] : read_row<PAIRS>(rows.x[i], lane); };
    auto d_of = [&](int i) { return EARLY ? dk[EARLY ? i : 0] : read_row<PAIRS>(rows.dh[i], lane); };
    auto fresh_of = [&](int i, int v) { return fresh<IO>(read_row<PAIRS>(rows.g[i], lane).at(v), a[i][v]); };
    auto advance = [&](int i, float (&y)[2]) {  // the state y after token i
      const Raw<IO> x = x_of(i);
#pragma unroll
      for (int v = 0; v < 2; ++v) y[v] = fmaf(a[i][v], y[v], COMPLEMENT ? fresh_of(i, v) * x.at(v) : x.at(v));
    };
    // the same for the rolled loops, from shared memory; their a and 1 - a of a token
    auto start = [&](int i, float (&y)[2]) { initial_of<PAIRS>(p, __shfl_sync(0xffffffffu, m.seq, i), l, y); };
    auto rolled_decay = [&](int i, float (&ai)[2], float (&ui)[2]) {
      const Raw<float> g = read_row<PAIRS>(rows.g[i], lane);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        ai[v] = decay<IO>(g.at(v));
        ui[v] = COMPLEMENT ? fresh<IO>(g.at(v), ai[v]) : 1.f;
      }
    };
    auto rolled = [&](int i, float (&y)[2]) {
      float ai[2], ui[2];
      rolled_decay(i, ai, ui);
      const Raw<IO> x = read_row<PAIRS>(rows.x[i], lane);
#pragma unroll
      for (int v = 0; v < 2; ++v) y[v] = fmaf(ai[v], y[v], COMPLEMENT ? ui[v] * x.at(v) : x.at(v));
    };
    auto end_gradient = [&](int i, float (&y)[2]) {  // what the end of a sequence brings
      const int sq = __shfl_sync(0xffffffffu, m.seq, i);
      y[0] = y[1] = 0.f;
      if (p.dfinal && l.any() && GDR_IN_BOUNDS(sq < p.num_seqs)) load2<PAIRS>(p.dfinal + (int64_t)sq * p.D, l, y);
    };
    if (!marked) {
#pragma unroll
      for (int i = 0; i < TOK; ++i) {
        const Raw<float> g = read_row<PAIRS>(rows.g[i], lane);
        if (EARLY) {
          xk[EARLY ? i : 0] = read_row<PAIRS>(rows.x[i], lane);
          dk[EARLY ? i : 0] = read_row<PAIRS>(rows.dh[i], lane);
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          a[i][v] = decay<IO>(g.at(v));
          gs[v] += g.at(v);
        }
      }
#pragma unroll
      for (int i = 0; i < TOK; ++i) advance(i, s);
#pragma unroll
      for (int i = TOK - 1; i >= 0; --i) {
        const Raw<IO> d = d_of(i);
#pragma unroll
        for (int v = 0; v < 2; ++v) r[v] = a[i][v] * (d.at(v) + r[v]);
      }
    } else {
      for (int i = 0; i < TOK; ++i) {
        if (m.first >> i & 1) start(i, s);
        rolled(i, s);
        const Raw<float> g = read_row<PAIRS>(rows.g[i], lane);
        gs[0] += g.at(0);
        gs[1] += g.at(1);
      }
      for (int i = TOK - 1; i >= 0; --i) {
        if (m.last >> i & 1) end_gradient(i, r);
        float ai[2], ui[2];
        rolled_decay(i, ai, ui);
        const Raw<IO> d = read_row<PAIRS>(rows.dh[i], lane);
#pragma unroll
        for (int v = 0; v < 2; ++v) r[v] = ai[v] * (d.at(v) + r[v]);
      }
    }
    {
      const float A[2] = {-expf(gs[0]), -expf(gs[1])};
      sh.map[buf][w][lane] = {{m.last ? kClosed : A[0], m.last ? kClosed : A[1]}, {r[0], r[1]}};
      states[w][lane] = {{m.first ? kClosed : A[0], m.first ? kClosed : A[1]}, {s[0], s[1]}};
    }
    if (__syncthreads_or(!alive)) return;  // a wait gave up; no copy is under way
    if (p.chained && w == 0 && q.in_group() != kGroup - 1) publish_tile<PAIRS, true>(p, sh, buf, q, l.c, lane);
    const Place nq = taken<true>(p, sh);
    const bool more = nq.step < p.tiles;
    if (EARLY && more && !marked) begin_copies<IO, PAIRS, true, TOK>(p, maps, rows, &sh.full[w], nq, w, lane);
    const bool next_marked = more && has_marks(p, nq.tile);
    enter_warp<false>(states, w, lane, h);
    r[0] = r[1] = 0.f;
    if (p.chained) {
      alive = enter_tile<PAIRS, true>(p, sh, buf, q, l.c, w, lane, r);
      if (!alive) l.on[0] = l.on[1] = false;  // writes nothing, and ends at the next barrier
    } else {
      __syncthreads();  // the next ticket is read before it is replaced
    }
    enter_warp<true>(sh.map[buf], w, lane, r);
    IO *dx0 = static_cast<IO *>(p.dx) + (int64_t)t0 * p.D;
    float *dg0 = p.dg + (int64_t)t0 * p.D;
    const int n = l.any() ? tokens_of<TOK>(p, t0) : 0;
    // from the carry r: dx, dg and the carry of the token before; `u` is 1 - a,
    // `past` h_{t-1}, less x_t for the complement
    auto write = [&](int i, const Raw<IO> &d, const float (&ai)[2], const float (&u)[2], const float (&past)[2]) {
      float dx[2], dg[2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float dt = d.at(v) + r[v];
        r[v] = ai[v] * dt;
        dx[v] = COMPLEMENT ? u[v] * dt : dt;
        dg[v] = r[v] * past[v];
      }
      if (i < n && GDR_IN_BOUNDS((int64_t)t0 + i < p.tokens)) {
        store2<PAIRS>(dx0 + (int64_t)i * p.D, l, dx);
        store2<PAIRS>(dg0 + (int64_t)i * p.D, l, dg);
      }
    };
    if (!marked) {
      float past[TOK][2];
#pragma unroll
      for (int i = 0; i < TOK; ++i) {
#pragma unroll
        for (int v = 0; v < 2; ++v) past[i][v] = COMPLEMENT ? h[v] - x_of(i).at(v) : h[v];
        if (i < TOK - 1) advance(i, h);
      }
#pragma unroll
      for (int i = TOK - 1; i >= 0; --i) {
        float u[2] = {1.f, 1.f};
        if (COMPLEMENT) {
          u[0] = fresh_of(i, 0);
          u[1] = fresh_of(i, 1);
        }
        write(i, d_of(i), a[i], u, past[i]);
      }
    } else {
      float past[TOK][2];  // (indexed by a running i: local memory)
      for (int i = 0; i < TOK; ++i) {
        if (m.first >> i & 1) start(i, h);
        const Raw<IO> x = read_row<PAIRS>(rows.x[i], lane);
#pragma unroll
        for (int v = 0; v < 2; ++v) past[i][v] = COMPLEMENT ? h[v] - x.at(v) : h[v];
        rolled(i, h);
      }
      for (int i = TOK - 1; i >= 0; --i) {
        if (m.last >> i & 1) end_gradient(i, r);
        float ai[2], ui[2];
        rolled_decay(i, ai, ui);
        write(i, read_row<PAIRS>(rows.dh[i], lane), ai, ui, past[i]);
        const int sq = __shfl_sync(0xffffffffu, m.seq, i);
        if (p.dinitial && (m.first >> i & 1) && l.any() && GDR_IN_BOUNDS(sq < p.num_seqs))
          store2<PAIRS>(p.dinitial + (int64_t)sq * p.D, l, r);
      }
    }
    if (q.tile == 0) pass_empty(p, p.dfinal, p.dinitial, false, q.stripe * kWide, kWide);
    if (!more) return;
    if (!EARLY || marked) begin_copies<IO, PAIRS, true, TOK>(p, maps, rows, &sh.full[w], nq, w, lane);
    marked = next_marked;
    q = nq;
  }
}

// Before the scan kernels: zeroes the ticket and the chain's words, checks the
// packed offsets, writes the status word and marks the tiles in which a
// sequence begins or ends.
__global__ void __launch_bounds__(256) glr_begin_kernel(GlrArgs p, int64_t words) {
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
      *p.status = bad ? KDA_DEVICE_BAD_CU_SEQLENS : KDA_DEVICE_OK;
      *p.ticket = 0;
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
  if (bad_offsets(p)) return;
  const int n = blockIdx.x;
  const int64_t r = backward ? n : state_row(p, n);
  if (r < 0) return;
  const float *src = backward ? p.dfinal : p.initial_state;
  float *dst = backward ? p.dinitial : p.final_state;
  for (int c = threadIdx.x; c < p.D; c += blockDim.x) dst[r * p.D + c] = src ? src[r * p.D + c] : 0.f;
}

// One token for each sequence, the state in place.
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

// A warp's rows of a [tokens, D] tensor: boxes of `tok` tokens x 64 channels, zeros outside.
bool make_map(CUtensorMap *m, const void *base, bool bf16, const GlrArgs &p, int64_t ld, int tok) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t e = bf16 ? 2 : 4;
  cuuint64_t dims[2] = {(cuuint64_t)p.D, (cuuint64_t)p.tokens}, strides[1] = {(cuuint64_t)ld * e};
  cuuint32_t box[2] = {kWide, (cuuint32_t)tok}, estr[2] = {1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
            const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

// The tiles of a launch with `tok` tokens a warp, and whether they wait for one
// another: not where each begins with a sequence's first token.
GlrArgs with_tiles(const GlrArgs &a, int tok) {
  GlrArgs p = a;
  p.tile_tokens = kWarps * tok;
  p.tiles = (p.tokens + p.tile_tokens - 1) / p.tile_tokens;
  p.stripes = (p.D + kWide - 1) / kWide;
  p.chained = p.tiles > 1 && (p.cu_seqlens || p.T > p.tile_tokens || p.tile_tokens % p.T != 0);
  p.groups = (p.tiles + kGroup - 1) / kGroup;
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
template <auto KERNEL>
cudaError_t launch_tiles(const char *name, size_t smem, const GlrArgs &p, const GlrMaps &maps, cudaStream_t s) {
  static std::atomic<int> cache[kCachedDevices];
  int most = 0;
  cudaError_t e = resident_blocks(KERNEL, cache, smem, &most);
  if (e != cudaSuccess) return e;
  const int64_t tiles = p.tiles * p.stripes;
  TraceScope tr(name, s);
  KERNEL<<<(unsigned)(tiles < most ? tiles : most), kThreads, smem, s>>>(p, maps);
  return cudaGetLastError();
}

template <typename IO, bool PAIRS, bool COMPLEMENT, bool STATES_ONLY>
cudaError_t launch_scan(const GlrArgs &a, cudaStream_t s) {
  constexpr int TOK = FwdShape<IO, PAIRS, COMPLEMENT>::kTok;
  const GlrArgs p = with_tiles(a, TOK);
  cudaError_t e = launch_begin(p, s);
  if (e != cudaSuccess) return e;
  if (p.tiles == 0) return launch_no_tokens(p, false, s);
  GlrMaps maps;
  if (PAIRS && !(make_map(&maps.x, p.x, p.bf16, p, p.ld_x, TOK) && make_map(&maps.g, p.g, false, p, p.ld_g, TOK)))
    return cudaErrorInvalidValue;
  return launch_tiles<glr_scan_kernel<IO, PAIRS, COMPLEMENT, STATES_ONLY>>(
      "glr_scan_kernel", kWarps * sizeof(WarpRows<IO, TOK>), p, maps, s);
}

template <typename IO, bool PAIRS, bool COMPLEMENT>
cudaError_t launch_fwd(const GlrArgs &a, cudaStream_t s) {
  return launch_scan<IO, PAIRS, COMPLEMENT, false>(a, s);
}

template <typename IO, bool PAIRS, bool COMPLEMENT>
cudaError_t launch_bwd(const GlrArgs &a, cudaStream_t s) {
  constexpr int TOK = BwdShape<IO, COMPLEMENT>::kTok;
  const GlrArgs p = with_tiles(a, TOK);
  cudaError_t e = cudaSuccess;
  if (p.own_chunks && p.tiles > 0) e = launch_scan<IO, PAIRS, COMPLEMENT, true>(a, s);
  if (e == cudaSuccess) e = launch_begin(p, s);
  if (e != cudaSuccess) return e;
  if (p.tiles == 0) return launch_no_tokens(p, true, s);
  GlrMaps maps;
  if (PAIRS && !(make_map(&maps.x, p.x, p.bf16, p, p.ld_x, TOK) && make_map(&maps.g, p.g, false, p, p.ld_g, TOK) &&
                 make_map(&maps.dh, p.dh, p.bf16, p, p.ld_dh, TOK)))
    return cudaErrorInvalidValue;
  return launch_tiles<glr_gradient_kernel<IO, PAIRS, COMPLEMENT>>(
      "glr_gradient_kernel", kWarps * sizeof(WarpRowsBwd<IO, TOK>), p, maps, s);
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
