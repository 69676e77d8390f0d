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
#include "common.cuh"
#include "internal.h"

namespace gdr {
namespace {

constexpr int kTile = kGlrChunk;  // tokens of a tile; a block's warps share them evenly

// V adjacent channels of one token, as they are read.
template <typename IO, int V> struct Raw;
template <> struct Raw<float, 1> {
  float r;
  __device__ __forceinline__ void zero() { r = 0.f; }
  __device__ __forceinline__ void load(const float *p) { r = __ldg(p); }
  __device__ __forceinline__ float at(int) const { return r; }
};
template <> struct Raw<float, 2> {
  float2 r;
  __device__ __forceinline__ void zero() { r = make_float2(0.f, 0.f); }
  __device__ __forceinline__ void load(const float *p) { r = __ldg(reinterpret_cast<const float2 *>(p)); }
  __device__ __forceinline__ float at(int v) const { return v ? r.y : r.x; }
};
template <> struct Raw<__nv_bfloat16, 1> {
  uint32_t r;
  __device__ __forceinline__ void zero() { r = 0; }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    r = __ldg(reinterpret_cast<const unsigned short *>(p));
  }
  __device__ __forceinline__ float at(int) const { return bf16_lo(r); }
};
template <> struct Raw<__nv_bfloat16, 2> {
  uint32_t r;
  __device__ __forceinline__ void zero() { r = 0; }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    r = __ldg(reinterpret_cast<const unsigned int *>(p));
  }
  __device__ __forceinline__ float at(int v) const { return v ? bf16_hi(r) : bf16_lo(r); }
};

template <typename IO, int V> __device__ __forceinline__ void store_row(IO *p, const float *x) {
  if constexpr (V == 1) io<IO>::store(p, x[0]);
  else if constexpr (sizeof(IO) == 4) *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
  else *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(x[0], x[1]);
}
// States are read and written in place by some calls: plain (coherent) accesses.
template <int V> __device__ __forceinline__ void load_state(const float *p, float *x) {
  if constexpr (V == 1) {
    x[0] = *p;
  } else {
    const float2 v = *reinterpret_cast<const float2 *>(p);
    x[0] = v.x; x[1] = v.y;
  }
}

// The decay of one token.  With bf16 activations the fast exponential: its error
// (2^-22 of the value) enters the state of a span of at most 16 tokens only,
// the decay of longer spans comes from the sum of their g.
template <typename IO> __device__ __forceinline__ float decay(float g) {
  if constexpr (sizeof(IO) == 2) return __expf(g);
  else return expf(g);
}

// Which of a warp's TOK tokens begin or end a sequence (bit i: token t0 + i), and,
// in lane i, the sequence of token t0 + i.
struct Marks {
  uint32_t first, last;
  int seq;
};
template <int TOK> __device__ __forceinline__ Marks find_marks(const GlrArgs &p, uint32_t t0, int lane) {
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
template <int V>
__device__ __forceinline__ void initial_of(const GlrArgs &p, int n, int c, bool on, float (&h0)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) h0[v] = 0.f;
  if (!p.initial_state) return;
  const int64_t r = state_row(p, n);
  if (on && r >= 0 && GDR_IN_BOUNDS(n < p.num_seqs && r < p.num_slots && c + V <= p.D))
    load_state<V>(p.initial_state + r * p.D + c, h0);
}

__device__ __forceinline__ bool bad_offsets(const GlrArgs &p) {
  return p.cu_seqlens && *reinterpret_cast<const volatile int32_t *>(p.status) != KDA_DEVICE_OK;
}

// Affine map of a span of tokens, for V channels: out = A in + H, or out = H
// where the span is closed.
template <int V> struct Map {
  float A[V], H[V];
  bool closed;
  __device__ __forceinline__ void identity() {
    closed = false;
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = 1.f; H[v] = 0.f; }
  }
  __device__ __forceinline__ float of(float in, int v) const { return closed ? H[v] : fmaf(A[v], in, H[v]); }
};

template <int V, int WARPS> struct TileShared {
  float G[WARPS][32 * V], A[WARPS][32 * V], H[WARPS][32 * V];     // per warp: sum of g, its exp, H
  float before_A[WARPS][32 * V], before_H[WARPS][32 * V];         // earlier tiles, a part a warp
  bool closed[WARPS], before_closed[WARPS];
  uint32_t ticket;
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
constexpr int kGroup = 16;
static_assert(kGroup >= kGlrShortestGroup, "the workspace counts groups of at least this length");
constexpr uint32_t kMaxChainPolls = 1u << 20;  // about a second

// A channel's map goes through the workspace as one 64-bit word, which is its
// own flag (no fence): H below, above it A with the sign bit set (A >= 0), or a
// code for a closed span.  0: not there yet.
constexpr uint32_t kClosedCode = 0xffbfffffu, kNanCode = 0xffffffffu;
__device__ __forceinline__ uint64_t pack_map(float A, float H, bool closed) {
  const uint32_t a = closed ? kClosedCode : A == A ? __float_as_uint(A) | 0x80000000u : kNanCode;
  return (uint64_t)a << 32 | __float_as_uint(H);
}
__device__ __forceinline__ bool word_closed(uint64_t u) { return (uint32_t)(u >> 32) == kClosedCode; }
__device__ __forceinline__ float word_A(uint64_t u) { return __uint_as_float((uint32_t)(u >> 32) & 0x7fffffffu); }
__device__ __forceinline__ float word_H(uint64_t u) { return __uint_as_float((uint32_t)u); }

template <int V> __device__ __forceinline__ void load_words(const uint64_t *p, uint64_t (&u)[V]) {
  if constexpr (V == 2)
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(u[0]), "=l"(u[1]) : "l"(p) : "memory");
  else
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(u[0]) : "l"(p) : "memory");
}
template <int V> __device__ __forceinline__ void store_words(uint64_t *p, const uint64_t (&u)[V]) {
  if constexpr (V == 2)
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p), "l"(u[0]), "l"(u[1]) : "memory");
  else
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(u[0]) : "memory");
}

// The place of a ticket's tile in the chain (REV: from the last tile on).
struct Place {
  uint32_t tile, step;  // its number on the token axis, and in the chain
  int stripe, in_group;
  uint32_t group;
};
template <bool REV> __device__ __forceinline__ Place place_of(const GlrArgs &p, uint32_t ticket) {
  Place q;
  q.step = ticket / (uint32_t)p.stripes;
  q.stripe = (int)(ticket - q.step * (uint32_t)p.stripes);
  q.tile = REV ? (uint32_t)p.tiles - 1 - q.step : q.step;
  q.group = q.step / kGroup;
  q.in_group = (int)(q.step % kGroup);
  return q;
}

// Publishes a tile's map, or what leaves its group (one warp, the tile's 32 V channels).
template <int V>
__device__ __forceinline__ void publish_map(const GlrArgs &p, const Place &q, const Map<V> &m, int c, bool on) {
  if (on && GDR_IN_BOUNDS(q.step < p.tiles && c + V <= p.D)) {
    uint64_t u[V];
#pragma unroll
    for (int v = 0; v < V; ++v) u[v] = pack_map(m.A[v], m.H[v], m.closed);
    store_words<V>(p.tile_map + (int64_t)q.step * p.pitch + c, u);
  }
}
template <int V>
__device__ __forceinline__ void publish_carry(const GlrArgs &p, const Place &q, const float (&h)[V], int c, bool on) {
  if (on && GDR_IN_BOUNDS(q.group < p.groups && c + V <= p.D)) {
    uint64_t u[V];
#pragma unroll
    for (int v = 0; v < V; ++v) u[v] = pack_map(0.f, h[v], true);
    store_words<V>(p.carry + (int64_t)q.group * p.pitch + c, u);
  }
}

// What enters the tile.  Each warp joins its part of the group's earlier maps
// (the first warp's part starts from what enters the group, a closed word), then
// all join the parts.  Every thread of the block takes part.  False: a wait gave up.
template <int V, int WARPS>
__device__ __forceinline__ bool enter_tile(const GlrArgs &p, TileShared<V, WARPS> &sh, const Place &q,
                                           int c, bool on, int w, int lane, float (&h)[V]) {
  constexpr int PER = kGroup / WARPS;  // maps a warp joins
  const int j0 = w * PER;
  const int n = on ? min(PER, q.in_group - j0) : 0;  // <= 0: none
  const bool start = on && w == 0 && q.group > 0;
  const uint64_t *maps = p.tile_map + (int64_t)(q.group * kGroup + j0) * p.pitch + c;
  const uint64_t *carry = p.carry + (int64_t)(q.group - 1) * p.pitch + c;
  uint64_t t[PER][V], s[V];
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) t[j][v] = 0;
  bool ok = false;
  for (uint32_t poll = 0; poll < kMaxChainPolls; ++poll) {
    // loads what is missing; a lane's channels come and go together or not
    bool have = true;
    if (start && (s[0] == 0 || s[V - 1] == 0) && GDR_IN_BOUNDS(q.group <= p.groups && c + V <= p.D)) load_words<V>(carry, s);
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (j < n && (t[j][0] == 0 || t[j][V - 1] == 0) && GDR_IN_BOUNDS(q.step < p.tiles && c + V <= p.D))
        load_words<V>(maps + (int64_t)j * p.pitch, t[j]);
    if (start) have = s[0] != 0 && s[V - 1] != 0;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (j < n) have = have && t[j][0] != 0 && t[j][V - 1] != 0;
    ok = __all_sync(0xffffffffu, have);
    if (ok) break;
    if ((poll & 1023) == 1023 && *reinterpret_cast<const volatile int32_t *>(p.status) != KDA_DEVICE_OK) break;
    if (poll == kMaxChainPolls - 1) *p.status = KDA_DEVICE_TIMEOUT;
  }
  Map<V> m;
  m.identity();
#pragma unroll
  for (int v = 0; v < V; ++v) m.H[v] = word_H(s[v]);
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (j < n) {
      const bool shut = word_closed(t[j][0]);
      m.closed |= shut;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        m.H[v] = shut ? word_H(t[j][v]) : fmaf(word_A(t[j][v]), m.H[v], word_H(t[j][v]));
        m.A[v] *= word_A(t[j][v]);
      }
    }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sh.before_A[w][lane * V + v] = m.A[v];
    sh.before_H[w][lane * V + v] = m.H[v];
  }
  if (lane == 0) sh.before_closed[w] = m.closed;
  if (__syncthreads_or(!ok)) return false;
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = sh.before_H[0][lane * V + v];
#pragma unroll
  for (int k = 1; k < WARPS; ++k)
    if (k * PER < q.in_group) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = sh.before_closed[k] ? sh.before_H[k][lane * V + v]
                                   : fmaf(sh.before_A[k][lane * V + v], h[v], sh.before_H[k][lane * V + v]);
    }
  return true;
}

// The map of the tile's tokens before warp w's (after them, for REV) from what
// the warps have shared.  Its decay is exp of the whole sum.
template <int V, int WARPS, bool REV>
__device__ __forceinline__ Map<V> map_before(const TileShared<V, WARPS> &sh, int w, int lane) {
  Map<V> m;
  m.identity();
  float gs[V];
#pragma unroll
  for (int v = 0; v < V; ++v) gs[v] = 0.f;
#pragma unroll
  for (int k = 0; k < WARPS; ++k) {
    const int j = REV ? WARPS - 1 - k : k;
    if (REV ? j > w : j < w) {
      m.closed |= sh.closed[j];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gs[v] += sh.G[j][lane * V + v];
        m.H[v] = sh.closed[j] ? sh.H[j][lane * V + v]
                              : fmaf(sh.A[j][lane * V + v], m.H[v], sh.H[j][lane * V + v]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) m.A[v] = expf(gs[v]);
  return m;
}

// Sequences without tokens, by the blocks of the first tile: what leaves them
// is what enters them.
template <int WARPS>
__device__ __forceinline__ void pass_empty(const GlrArgs &p, const float *src, float *dst, bool pooled,
                                           int c0, int width) {
  if (!dst || !p.cu_seqlens) return;
  const int lane = threadIdx.x & 31;
  for (int n0 = (threadIdx.x >> 5) * 32; n0 < p.num_seqs; n0 += WARPS * 32) {
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
  const uint32_t t = tile * kTile, r = t % (uint32_t)p.T;
  return r == 0 || r + kTile >= (uint32_t)p.T;
}

// ---- forward ------------------------------------------------------------
template <typename IO, int V, int TOK> struct Tokens {
  Raw<IO, V> x[TOK];
  Raw<float, V> g[TOK];
  bool marked;
  __device__ __forceinline__ void load(const GlrArgs &p, uint32_t tile, uint32_t t0, int c, bool on) {
    const IO *x0 = static_cast<const IO *>(p.x) + (int64_t)t0 * p.ld_x + c;
    const float *g0 = p.g + (int64_t)t0 * p.ld_g + c;
    const int n = on ? (int)min((int64_t)TOK, p.tokens - t0) : 0;
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      x[i].zero();
      g[i].zero();
      if (i < n && GDR_IN_BOUNDS(t0 + i < p.tokens && c + V <= p.D)) {
        x[i].load(x0 + i * p.ld_x);
        g[i].load(g0 + i * p.ld_g);
      }
    }
    marked = has_marks(p, tile);
  }
};

// Persistent blocks: the loads of a block's next tile are under way while this
// one waits for what enters it and is written.  x and g are read once; the
// tokens' a stays in registers in between.  STATES_ONLY: only the saved chunk
// states are written.
template <typename IO, int V, bool COMPLEMENT, bool STATES_ONLY>
__global__ void __launch_bounds__(128, 4) glr_scan_kernel(GlrArgs p) {
  constexpr int WARPS = 4, TOK = kTile / WARPS;
  __shared__ TileShared<V, WARPS> sh;
  if (bad_offsets(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t total = (uint32_t)(p.tiles * p.stripes);
  if (threadIdx.x == 0) sh.ticket = p.chained ? (uint32_t)atomicAdd(p.ticket, 1) : blockIdx.x;
  __syncthreads();
  uint32_t ticket = sh.ticket;
  __syncthreads();
  if (ticket >= total) return;
  Place q = place_of<false>(p, ticket);
  Tokens<IO, V, TOK> k;
  {
    const int c = (q.stripe * 32 + lane) * V;
    k.load(p, q.tile, q.tile * kTile + w * TOK, c, c < p.D);
  }
  while (true) {
    if (threadIdx.x == 0) sh.ticket = p.chained ? (uint32_t)atomicAdd(p.ticket, 1) : ticket + gridDim.x;
    const uint32_t t0 = q.tile * kTile + w * TOK;
    const int c = (q.stripe * 32 + lane) * V;
    const bool on = c < p.D;
    Marks m;
    m.first = m.last = 0;
    m.seq = 0;
    if (k.marked) m = find_marks<TOK>(p, t0, lane);
    // the span from zeros; b of a token is x, or (1 - a) x
    float a[TOK][V], b[COMPLEMENT ? TOK : 1][V], gs[V], h[V];
    Raw<IO, V> x[TOK];
#pragma unroll
    for (int v = 0; v < V; ++v) gs[v] = h[v] = 0.f;
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      x[i] = k.x[i];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float g = k.g[i].at(v);
        a[i][v] = decay<IO>(g);
        if (COMPLEMENT) b[i][v] = -expm1f(g) * x[i].at(v);
        gs[v] += g;
      }
    }
    auto b_of = [&](int i, int v) { return COMPLEMENT ? b[COMPLEMENT ? i : 0][v] : x[i].at(v); };
    if (m.first == 0) {
#pragma unroll
      for (int i = 0; i < TOK; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(a[i][v], h[v], b_of(i, v));
    } else {
#pragma unroll
      for (int i = 0; i < TOK; ++i) {
        if (m.first >> i & 1) {
          // a start's state takes the place of its a: the initial state is read
          // once, before the map is published (the sequence's last tile may
          // write the final state over it as soon as that is done)
          float h0[V];
          initial_of<V>(p, __shfl_sync(0xffffffffu, m.seq, i), c, on, h0);
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = a[i][v] = fmaf(a[i][v], h0[v], b_of(i, v));
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = fmaf(a[i][v], h[v], b_of(i, v));
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      sh.G[w][lane * V + v] = gs[v];
      sh.A[w][lane * V + v] = expf(gs[v]);
      sh.H[w][lane * V + v] = h[v];
    }
    if (lane == 0) sh.closed[w] = m.first != 0;
    __syncthreads();
    // the next tile's loads
    const uint32_t next = sh.ticket;
    const Place nq = place_of<false>(p, next < total ? next : 0);
    {
      const int nc = (nq.stripe * 32 + lane) * V;
      k.load(p, nq.tile, nq.tile * kTile + w * TOK, nc, next < total && nc < p.D);
    }
    const bool group_end = q.in_group == kGroup - 1;
    if (p.chained && w == WARPS - 1 && !group_end)
      publish_map<V>(p, q, map_before<V, WARPS, false>(sh, WARPS, lane), c, on);
    const Map<V> before = map_before<V, WARPS, false>(sh, w, lane);
    float in[V];
#pragma unroll
    for (int v = 0; v < V; ++v) in[v] = 0.f;
    if (p.chained) {
      if (!enter_tile<V, WARPS>(p, sh, q, c, on, w, lane, in)) return;
    } else {
      __syncthreads();  // the maps are read before the next tile's are written
    }
    if (w == 0 && on && p.chunk_states && GDR_IN_BOUNDS(q.tile < p.tiles && c + V <= p.D))
      store_row<float, V>(p.chunk_states + (int64_t)q.tile * p.D + c, in);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = before.of(in[v], v);
    if (p.chained && w == WARPS - 1 && group_end) {
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v)
        out[v] = m.first ? sh.H[w][lane * V + v] : fmaf(sh.A[w][lane * V + v], h[v], sh.H[w][lane * V + v]);
      publish_carry<V>(p, q, out, c, on);
    }
    if (!STATES_ONLY) {
      IO *out = static_cast<IO *>(p.h) + (int64_t)t0 * p.D + c;
      const int n = on ? (int)min((int64_t)TOK, p.tokens - t0) : 0;
      if ((m.first | m.last) == 0) {
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = fmaf(a[i][v], h[v], b_of(i, v));
          if (i < n && GDR_IN_BOUNDS(t0 + i < p.tokens && c + V <= p.D)) store_row<IO, V>(out + (int64_t)i * p.D, h);
        }
      } else {
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
          const int s = __shfl_sync(0xffffffffu, m.seq, i);
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = m.first >> i & 1 ? a[i][v] : fmaf(a[i][v], h[v], b_of(i, v));
          if (i < n && GDR_IN_BOUNDS(t0 + i < p.tokens && c + V <= p.D)) store_row<IO, V>(out + (int64_t)i * p.D, h);
          if ((m.last >> i & 1) && p.final_state) {
            const int64_t r = state_row(p, s);
            if (on && r >= 0 && GDR_IN_BOUNDS(s < p.num_seqs && r < p.num_slots && c + V <= p.D))
              store_row<float, V>(p.final_state + r * p.D + c, h);
          }
        }
      }
      if (q.tile == 0) pass_empty<WARPS>(p, p.initial_state, p.final_state, true, q.stripe * 32 * V, 32 * V);
    }
    if (next >= total) return;
    ticket = next;
    q = nq;
  }
}

// ---- backward -----------------------------------------------------------
// The states again from what enters the tile (saved), the gradients from what
// enters it from the tokens after it (chained): x, g and dh are read once.
template <typename IO, int V, bool COMPLEMENT>
__global__ void __launch_bounds__(256, 2) glr_gradient_kernel(GlrArgs p) {
  constexpr int WARPS = 8, TOK = kTile / WARPS;
  __shared__ TileShared<V, WARPS> sh;
  __shared__ float state_H[WARPS][32 * V];
  __shared__ bool state_closed[WARPS];
  if (bad_offsets(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t total = (uint32_t)(p.tiles * p.stripes);
  if (threadIdx.x == 0) sh.ticket = p.chained ? (uint32_t)atomicAdd(p.ticket, 1) : blockIdx.x;
  __syncthreads();
  uint32_t ticket = sh.ticket;
  __syncthreads();
  if (ticket >= total) return;
  Place q = place_of<true>(p, ticket);
  Tokens<IO, V, TOK> k;
  Raw<IO, V> kd[TOK];
  float kh[V];
  auto load = [&](const Place &at, bool live) {
    const uint32_t t0 = at.tile * kTile + w * TOK;
    const int c = (at.stripe * 32 + lane) * V;
    const bool on = live && c < p.D;
    k.load(p, at.tile, t0, c, on);
    const IO *d0 = static_cast<const IO *>(p.dh) + (int64_t)t0 * p.ld_dh + c;
    const int n = on ? (int)min((int64_t)TOK, p.tokens - t0) : 0;
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      kd[i].zero();
      if (i < n && GDR_IN_BOUNDS(t0 + i < p.tokens && c + V <= p.D)) kd[i].load(d0 + i * p.ld_dh);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) kh[v] = 0.f;
    if (on && GDR_IN_BOUNDS(at.tile < p.tiles && c + V <= p.D))
      load_state<V>(p.chunk_states + (int64_t)at.tile * p.D + c, kh);
  };
  load(q, true);
  while (true) {
    if (threadIdx.x == 0) sh.ticket = p.chained ? (uint32_t)atomicAdd(p.ticket, 1) : ticket + gridDim.x;
    const uint32_t t0 = q.tile * kTile + w * TOK;
    const int c = (q.stripe * 32 + lane) * V;
    const bool on = c < p.D;
    Marks m;
    m.first = m.last = 0;
    m.seq = 0;
    if (k.marked) m = find_marks<TOK>(p, t0, lane);
    float a[TOK][V], u[COMPLEMENT ? TOK : 1][V], x[TOK][V], d[TOK][V], gs[V], s[V], qv[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      gs[v] = s[v] = qv[v] = 0.f;
      h[v] = kh[v];
    }
#pragma unroll
    for (int i = 0; i < TOK; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float g = k.g[i].at(v);
        a[i][v] = decay<IO>(g);
        if (COMPLEMENT) u[i][v] = -expm1f(g);
        x[i][v] = k.x[i].at(v);
        d[i][v] = kd[i].at(v);
        gs[v] += g;
      }
    auto b_of = [&](int i, int v) { return COMPLEMENT ? u[COMPLEMENT ? i : 0][v] * x[i][v] : x[i][v]; };
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      if (m.first >> i & 1) initial_of<V>(p, __shfl_sync(0xffffffffu, m.seq, i), c, on, s);
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = fmaf(a[i][v], s[v], b_of(i, v));
    }
#pragma unroll
    for (int i = TOK - 1; i >= 0; --i) {
      if (m.last >> i & 1) {  // the gradient of the sequence's final state enters here
        const int n = __shfl_sync(0xffffffffu, m.seq, i);
        float df[V];
#pragma unroll
        for (int v = 0; v < V; ++v) df[v] = 0.f;
        if (p.dfinal && on && GDR_IN_BOUNDS(n < p.num_seqs && c + V <= p.D))
          load_state<V>(p.dfinal + (int64_t)n * p.D + c, df);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          d[i][v] += df[v];
          qv[v] = 0.f;
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) qv[v] = a[i][v] * (d[i][v] + qv[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      sh.G[w][lane * V + v] = gs[v];
      sh.A[w][lane * V + v] = expf(gs[v]);
      sh.H[w][lane * V + v] = qv[v];
      state_H[w][lane * V + v] = s[v];
    }
    if (lane == 0) {
      sh.closed[w] = m.last != 0;
      state_closed[w] = m.first != 0;
    }
    __syncthreads();
    const uint32_t next = sh.ticket;
    const Place nq = place_of<true>(p, next < total ? next : 0);
    load(nq, next < total);
#pragma unroll
    for (int j = 0; j < WARPS - 1; ++j)  // the state that enters the warp
      if (j < w)
#pragma unroll
        for (int v = 0; v < V; ++v)
          h[v] = state_closed[j] ? state_H[j][lane * V + v]
                                 : fmaf(sh.A[j][lane * V + v], h[v], state_H[j][lane * V + v]);
    const bool group_end = q.in_group == kGroup - 1;
    if (p.chained && w == 0 && !group_end)
      publish_map<V>(p, q, map_before<V, WARPS, true>(sh, -1, lane), c, on);
    const Map<V> after = map_before<V, WARPS, true>(sh, w, lane);
    float in[V];
#pragma unroll
    for (int v = 0; v < V; ++v) in[v] = 0.f;
    if (p.chained) {
      if (!enter_tile<V, WARPS>(p, sh, q, c, on, w, lane, in)) return;
    } else {
      __syncthreads();  // the maps are read before the next tile's are written
    }
#pragma unroll
    for (int v = 0; v < V; ++v) qv[v] = after.of(in[v], v);
    if (p.chained && w == 0 && group_end) {
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v)
        out[v] = m.last ? sh.H[w][lane * V + v] : fmaf(sh.A[w][lane * V + v], qv[v], sh.H[w][lane * V + v]);
      publish_carry<V>(p, q, out, c, on);
    }
    float before[TOK][V];  // h_{t-1}
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      if (m.first >> i & 1) initial_of<V>(p, __shfl_sync(0xffffffffu, m.seq, i), c, on, h);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        before[i][v] = COMPLEMENT ? h[v] - x[i][v] : h[v];
        h[v] = fmaf(a[i][v], h[v], b_of(i, v));
      }
    }
    IO *dx0 = static_cast<IO *>(p.dx) + (int64_t)t0 * p.D + c;
    float *dg0 = p.dg + (int64_t)t0 * p.D + c;
    const int n = on ? (int)min((int64_t)TOK, p.tokens - t0) : 0;
#pragma unroll
    for (int i = TOK - 1; i >= 0; --i) {
      float dx[V], dg[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float dt = m.last >> i & 1 ? d[i][v] : d[i][v] + qv[v];
        qv[v] = a[i][v] * dt;
        dx[v] = COMPLEMENT ? u[COMPLEMENT ? i : 0][v] * dt : dt;
        dg[v] = qv[v] * before[i][v];
      }
      if (i < n && GDR_IN_BOUNDS(t0 + i < p.tokens && c + V <= p.D)) {
        store_row<IO, V>(dx0 + (int64_t)i * p.D, dx);
        store_row<float, V>(dg0 + (int64_t)i * p.D, dg);
      }
      if (p.dinitial && (m.first >> i & 1)) {
        const int sq = __shfl_sync(0xffffffffu, m.seq, i);
        if (on && GDR_IN_BOUNDS(sq < p.num_seqs && c + V <= p.D))
          store_row<float, V>(p.dinitial + (int64_t)sq * p.D + c, qv);
      }
    }
    if (q.tile == 0) pass_empty<WARPS>(p, p.dfinal, p.dinitial, false, q.stripe * 32 * V, 32 * V);
    if (next >= total) return;
    ticket = next;
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
      const int64_t t = tile * kTile;
      int lo = 0, hi = p.num_seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_seqlens[mid] <= t) lo = mid;
        else hi = mid;
      }
      p.tile_marks[tile] = p.cu_seqlens[lo] == t || p.cu_seqlens[lo + 1] <= t + kTile;
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
template <typename IO, int V, bool COMPLEMENT>
__global__ void __launch_bounds__(256) glr_step_kernel(GlrArgs p) {
  const int c = (blockIdx.x * 256 + threadIdx.x) * V;
  if (c >= p.D) return;
  for (int n = blockIdx.y; n < p.num_seqs; n += gridDim.y) {
    const int64_t r = state_row(p, n);
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
    if (r >= 0 && GDR_IN_BOUNDS(r < p.num_slots && c + V <= p.D)) {
      Raw<IO, V> x;
      Raw<float, V> g;
      x.load(static_cast<const IO *>(p.x) + n * p.ld_x + c);
      g.load(p.g + n * p.ld_g + c);
      load_state<V>(p.final_state + r * p.D + c, h);
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = fmaf(expf(g.at(v)), h[v], COMPLEMENT ? -expm1f(g.at(v)) * x.at(v) : x.at(v));
      store_row<float, V>(p.final_state + r * p.D + c, h);
    }
    if (GDR_IN_BOUNDS(c + V <= p.D)) store_row<IO, V>(static_cast<IO *>(p.h) + (int64_t)n * p.D + c, h);
  }
}

bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Two channels a lane where rows and pointers allow 2-channel accesses, else one.
bool pairs_ok(const GlrArgs &p) {
  const size_t e = p.bf16 ? 2 : 4;
  return p.D % 2 == 0 && p.ld_x % 2 == 0 && p.ld_g % 2 == 0 && p.ld_dh % 2 == 0 &&
         aligned_to(p.x, 2 * e) && aligned_to(p.h, 2 * e) && aligned_to(p.dh, 2 * e) &&
         aligned_to(p.dx, 2 * e) && aligned_to(p.g, 8) && aligned_to(p.dg, 8) &&
         aligned_to(p.initial_state, 8) && aligned_to(p.final_state, 8) &&
         aligned_to(p.dinitial, 8) && aligned_to(p.chunk_states, 8);
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

// The stripes of a call, and whether its tiles wait for one another: not where
// each begins with a sequence's first token.
template <int V> GlrArgs with_chain(const GlrArgs &a) {
  GlrArgs p = a;
  p.stripes = (p.D + 32 * V - 1) / (32 * V);
  p.chained = p.tiles > 1 && (p.cu_seqlens || p.T > kTile || kTile % p.T != 0);
  p.groups = (p.tiles + kGroup - 1) / kGroup;
  p.carry = p.tile_map + p.tiles * p.pitch;
  return p;
}

// As many blocks as run at once, or one a tile.
unsigned persistent_grid(const GlrArgs &p, int per_sm) {
  const int64_t tiles = p.tiles * p.stripes, most = (int64_t)sm_count() * per_sm;
  return (unsigned)(tiles < most ? tiles : most);
}

template <typename IO, int V, bool COMPLEMENT>
cudaError_t launch_fwd(const GlrArgs &a, cudaStream_t s) {
  const GlrArgs p = with_chain<V>(a);
  cudaError_t e = launch_begin(p, s);
  if (e != cudaSuccess) return e;
  if (p.tiles == 0) return launch_no_tokens(p, false, s);
  TraceScope tr("glr_scan_kernel", s);
  glr_scan_kernel<IO, V, COMPLEMENT, false><<<persistent_grid(p, 4), 128, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename IO, int V, bool COMPLEMENT>
cudaError_t launch_bwd(const GlrArgs &a, cudaStream_t s) {
  const GlrArgs p = with_chain<V>(a);
  cudaError_t e = launch_begin(p, s);
  if (e != cudaSuccess) return e;
  if (p.tiles == 0) return launch_no_tokens(p, true, s);
  if (p.own_chunks) {
    {
      TraceScope tr("glr_scan_kernel", s);
      glr_scan_kernel<IO, V, COMPLEMENT, true><<<persistent_grid(p, 4), 128, 0, s>>>(p);
    }
    e = launch_begin(p, s);
    if (e != cudaSuccess) return e;
  }
  TraceScope tr("glr_gradient_kernel", s);
  glr_gradient_kernel<IO, V, COMPLEMENT><<<persistent_grid(p, 2), 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename IO, int V, bool COMPLEMENT>
cudaError_t launch_step(const GlrArgs &p, cudaStream_t s) {
  TraceScope tr("glr_step_kernel", s);
  const dim3 grid((unsigned)((p.D + 256 * V - 1) / (256 * V)),
                  (unsigned)(p.num_seqs < 65535 ? p.num_seqs : 65535));
  glr_step_kernel<IO, V, COMPLEMENT><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

#define GDR_GLR_DISPATCH(fn)                                                            \
  do {                                                                                  \
    const bool two = pairs_ok(p);                                                       \
    if (p.bf16)                                                                         \
      return p.complement ? (two ? fn<__nv_bfloat16, 2, true>(p, s) : fn<__nv_bfloat16, 1, true>(p, s))   \
                          : (two ? fn<__nv_bfloat16, 2, false>(p, s) : fn<__nv_bfloat16, 1, false>(p, s)); \
    return p.complement ? (two ? fn<float, 2, true>(p, s) : fn<float, 1, true>(p, s))   \
                        : (two ? fn<float, 2, false>(p, s) : fn<float, 1, false>(p, s)); \
  } while (0)

}  // namespace

GDR_DEFINE_OOB_COUNTER(oob_count_glr)

cudaError_t launch_glr_fwd(const GlrArgs &p, cudaStream_t s) { GDR_GLR_DISPATCH(launch_fwd); }
cudaError_t launch_glr_bwd(const GlrArgs &p, cudaStream_t s) { GDR_GLR_DISPATCH(launch_bwd); }
cudaError_t launch_glr_step(const GlrArgs &p, cudaStream_t s) { GDR_GLR_DISPATCH(launch_step); }

}  // namespace gdr
