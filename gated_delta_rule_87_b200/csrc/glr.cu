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

constexpr int kTok = 8;                    // tokens of a warp
constexpr int kScanWarps = 8;              // warps of a block
constexpr int kTile = kTok * kScanWarps;   // tokens of a tile
static_assert(kTile == kGlrChunk, "a tile is a chunk");

// V adjacent channels of one row.
template <typename IO, int V> struct row;
template <typename IO> struct row<IO, 1> {
  static __device__ __forceinline__ void load(const IO *p, float *x) { x[0] = io<IO>::load(p); }
  static __device__ __forceinline__ void store(IO *p, const float *x) { io<IO>::store(p, x[0]); }
};
template <> struct row<float, 2> {
  static __device__ __forceinline__ void load(const float *p, float *x) {
    const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
    x[0] = v.x; x[1] = v.y;
  }
  static __device__ __forceinline__ void store(float *p, const float *x) {
    *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
  }
};
template <> struct row<__nv_bfloat16, 2> {
  static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float *x) {
    const uint32_t u = __ldg(reinterpret_cast<const unsigned int *>(p));
    x[0] = bf16_lo(u); x[1] = bf16_hi(u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *x) {
    *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(x[0], x[1]);
  }
};

// States are read and written in place by some calls: plain (coherent) accesses.
template <int V> __device__ __forceinline__ void state_load(const float *p, float *x) {
  if constexpr (V == 2) {
    const float2 v = *reinterpret_cast<const float2 *>(p);
    x[0] = v.x; x[1] = v.y;
  } else {
    x[0] = *p;
  }
}

// Which of a warp's tokens begin or end a sequence (bit i: token t0 + i), and,
// in lane i, the sequence of token t0 + i.
struct Marks {
  uint32_t first, last;
  int seq;
};
__device__ __forceinline__ Marks find_marks(const GlrArgs &p, int64_t t0, int lane) {
  Marks m;
  bool f = false, l = false;
  m.seq = 0;
  const int64_t t = t0 + lane;
  if (lane < kTok && t < p.tokens) {
    if (p.cu_seqlens) {  // the last sequence that starts at or before t (empty ones start there too)
      int lo = 0, hi = p.num_seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu_seqlens + mid) <= t) lo = mid;
        else hi = mid;
      }
      m.seq = lo;
      f = __ldg(p.cu_seqlens + lo) == t;
      l = __ldg(p.cu_seqlens + lo + 1) == t + 1;
    } else {
      m.seq = (int)(t / p.T);
      const int64_t r = t - (int64_t)m.seq * p.T;
      f = r == 0;
      l = r == p.T - 1;
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

__device__ __forceinline__ bool bad_offsets(const GlrArgs &p) {
  return p.cu_seqlens && *reinterpret_cast<const volatile int32_t *>(p.status) != KDA_DEVICE_OK;
}

// One warp's tokens: per token the decay a, the gate value g and the input x.
template <typename IO, int V>
__device__ __forceinline__ void load_tokens(const GlrArgs &p, int64_t t0, int c, bool on,
                                            float (&x)[kTok][V], float (&g)[kTok][V]) {
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[i][v] = g[i][v] = 0.f;
    const int64_t t = t0 + i;
    if (on && t < p.tokens && GDR_IN_BOUNDS(c + V <= p.D)) {
      row<IO, V>::load(static_cast<const IO *>(p.x) + t * p.ld_x + c, x[i]);
      row<float, V>::load(p.g + t * p.ld_g + c, g[i]);
    }
  }
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
  // this span, then the one of (a, h, c)
  __device__ __forceinline__ void then(const float (&a)[V], const float (&h)[V], bool c) {
    closed |= c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      H[v] = c ? h[v] : fmaf(a[v], H[v], h[v]);
      A[v] *= a[v];
    }
  }
  __device__ __forceinline__ float of(float in, int v) const { return closed ? H[v] : fmaf(A[v], in, H[v]); }
};

template <int V> struct TileShared {
  float G[kScanWarps][32 * V], A[kScanWarps][32 * V], H[kScanWarps][32 * V];  // per warp: sum of g, its exp, H
  float before_A[kScanWarps][32 * V], before_H[kScanWarps][32 * V];           // earlier tiles, a part a warp
  bool closed[kScanWarps], before_closed[kScanWarps];
  int ticket;
};

// ---- the chain of tiles -------------------------------------------------
// Tiles are taken in order of a ticket, so every tile that another waits for
// has been taken by a block that runs or has ended.  Groups of `group` tiles:
// a tile publishes its map as soon as it has it; what enters a tile is what
// enters its group, through the maps of the group's tiles before it; the last
// tile of a group publishes what leaves the group.  Which values are joined,
// and in which order, depends on the sizes alone, never on timing.
constexpr int kMapOpen = 1, kMapClosed = 2;
constexpr uint32_t kMaxChainPolls = 1u << 20;  // about a second

__device__ __forceinline__ int load_acquire(const int32_t *p) {
  int v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(int32_t *p, int v) {
  asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Waits for a flag; 0 if it gave up (or another block did: the status word says so).
__device__ __forceinline__ int wait_flag(const GlrArgs &p, const int32_t *flag) {
  for (uint32_t i = 0; i < kMaxChainPolls; ++i) {
    const int v = load_acquire(flag);
    if (v) return v;
    if ((i & 1023) == 1023 && load_acquire(p.status) != KDA_DEVICE_OK) return 0;
  }
  *p.status = KDA_DEVICE_TIMEOUT;
  return 0;
}

// The place of a tile in the chain (REV: from the last tile on).
struct Place {
  int64_t tile, step;  // its number on the token axis, and in the chain
  int stripe, in_group;
  int64_t group;
};
template <bool REV> __device__ __forceinline__ Place place_of(const GlrArgs &p, int64_t ticket) {
  Place q;
  q.step = ticket / p.stripes;
  q.stripe = (int)(ticket - q.step * p.stripes);
  q.tile = REV ? p.tiles - 1 - q.step : q.step;
  q.group = q.step / p.group;
  q.in_group = (int)(q.step - q.group * p.group);
  return q;
}

// The block's tile: a ticket where tiles wait for one another, else the block's number.
template <int V> __device__ __forceinline__ int64_t take_tile(const GlrArgs &p, TileShared<V> &sh) {
  if (!p.chained) return blockIdx.x;
  if (threadIdx.x == 0) sh.ticket = atomicAdd(p.ticket, 1);
  __syncthreads();
  return sh.ticket;
}

// Publishes a tile's map (one warp, the tile's 32 V channels).
template <int V>
__device__ __forceinline__ void publish_map(const GlrArgs &p, const Place &q, const Map<V> &m, int c,
                                            bool on, int lane) {
  if (on && GDR_IN_BOUNDS(q.step < p.tiles && c + V <= p.D)) {
    float2 *to = reinterpret_cast<float2 *>(p.tile_map) + q.step * p.D + c;
#pragma unroll
    for (int v = 0; v < V; ++v) __stcg(to + v, make_float2(m.A[v], m.H[v]));
  }
  __threadfence();
  __syncwarp();
  if (lane == 0) store_release(p.tile_flag + q.step * p.stripes + q.stripe, m.closed ? kMapClosed : kMapOpen);
}
template <int V>
__device__ __forceinline__ void publish_carry(const GlrArgs &p, const Place &q, const float (&h)[V],
                                              int c, bool on, int lane) {
  if (on && GDR_IN_BOUNDS(q.group < p.groups && c + V <= p.D)) {
#pragma unroll
    for (int v = 0; v < V; ++v) __stcg(p.carry + q.group * p.D + c + v, h[v]);
  }
  __threadfence();
  __syncwarp();
  if (lane == 0) store_release(p.carry_flag + q.group * p.stripes + q.stripe, kMapOpen);
}

// What enters the tile.  Each warp joins its part of the group's earlier maps,
// then all join the parts.  Every thread of the block takes part.  False: a wait gave up.
template <int V>
__device__ __forceinline__ bool enter_tile(const GlrArgs &p, TileShared<V> &sh, const Place &q, int c,
                                           bool on, int w, int lane, float (&h)[V]) {
  const int per = p.group / kScanWarps;  // maps a warp joins, 1 to 4
  Map<V> m;
  m.identity();
  float carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = 0.f;
  bool ok = true;
  const int j0 = w * per;
  const int n = min(per, q.in_group - j0);  // <= 0: none
  const int64_t first = q.group * p.group + j0;
  int flag = kMapOpen;
  if (lane < n) flag = wait_flag(p, p.tile_flag + (first + lane) * p.stripes + q.stripe);
  // the group's start is needed by whoever joins the parts; warp 0 has the most time for it
  if (w == 0 && lane == 31 && q.group > 0)
    flag = wait_flag(p, p.carry_flag + (q.group - 1) * p.stripes + q.stripe);
  ok = __all_sync(0xffffffffu, flag != 0);
  const uint32_t closed = __ballot_sync(0xffffffffu, flag == kMapClosed);
  if (ok && n > 0) {
    float2 t[4][V];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        t[j][v] = make_float2(1.f, 0.f);
        if (j < n && on && GDR_IN_BOUNDS(first + j < p.tiles && c + V <= p.D))
          t[j][v] = __ldcg(reinterpret_cast<const float2 *>(p.tile_map) + (first + j) * p.D + c + v);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a[V], hh[V];
#pragma unroll
      for (int v = 0; v < V; ++v) { a[v] = t[j][v].x; hh[v] = t[j][v].y; }
      if (j < n) m.then(a, hh, closed >> j & 1);
    }
  }
  if (ok && w == 0 && q.group > 0 && on && GDR_IN_BOUNDS(q.group <= p.groups))
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = __ldcg(p.carry + (q.group - 1) * p.D + c + v);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // warp 0's part starts from what enters the group
    if (w == 0) m.H[v] = m.of(carry[v], v);
    sh.before_A[w][lane * V + v] = m.A[v];
    sh.before_H[w][lane * V + v] = m.H[v];
  }
  if (lane == 0) sh.before_closed[w] = m.closed;
  if (__syncthreads_or(!ok)) return false;
  const int parts = min(kScanWarps, (q.in_group + per - 1) / per);
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = sh.before_H[0][lane * V + v];
  for (int k = 1; k < parts; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v)
      h[v] = sh.before_closed[k] ? sh.before_H[k][lane * V + v]
                                 : fmaf(sh.before_A[k][lane * V + v], h[v], sh.before_H[k][lane * V + v]);
  return true;
}

// A warp's map goes to shared memory ...
template <int V>
__device__ __forceinline__ void share_map(float (&G)[32 * V], float (&A)[32 * V], float (&H)[32 * V],
                                          int lane, const float (&gs)[V], const float (&h)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    G[lane * V + v] = gs[v];
    A[lane * V + v] = expf(gs[v]);
    H[lane * V + v] = h[v];
  }
}
// ... and this is the map of the tile's tokens before warp w's (after them, for
// REV).  Its decay is exp of the whole sum.
template <int V, bool REV>
__device__ __forceinline__ Map<V> map_before(const TileShared<V> &sh, int w, int lane) {
  Map<V> m;
  m.identity();
  float gs[V];
#pragma unroll
  for (int v = 0; v < V; ++v) gs[v] = 0.f;
#pragma unroll
  for (int k = 0; k < kScanWarps; ++k) {
    const int j = REV ? kScanWarps - 1 - k : k;
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
__device__ __forceinline__ void pass_empty(const GlrArgs &p, const float *src, float *dst, bool pooled,
                                           int c0, int width) {
  if (!dst || !p.cu_seqlens) return;
  const int lane = threadIdx.x & 31;
  for (int n0 = (threadIdx.x >> 5) * 32; n0 < p.num_seqs; n0 += kScanWarps * 32) {
    const int n = n0 + lane;
    const bool empty = n < p.num_seqs && __ldg(p.cu_seqlens + n) == __ldg(p.cu_seqlens + n + 1);
    uint32_t todo = __ballot_sync(0xffffffffu, empty);
    while (todo) {
      const int k = n0 + __ffs(todo) - 1;
      todo &= todo - 1;
      const int64_t r = pooled ? state_row(p, k) : k;
      if (r < 0) continue;
      for (int c = c0 + lane; c < c0 + width && c < p.D; c += 32) dst[r * p.D + c] = src ? src[r * p.D + c] : 0.f;
    }
  }
}

// b_t of a warp's tokens, with the initial state folded in at a sequence's
// first token: there h = a h0 + b, and nothing before it counts.
template <int V, bool COMPLEMENT>
__device__ __forceinline__ void make_inputs(const GlrArgs &p, const Marks &m, int c, bool on,
                                            const float (&x)[kTok][V], const float (&g)[kTok][V],
                                            float (&a)[kTok][V], float (&b)[kTok][V]) {
#pragma unroll
  for (int i = 0; i < kTok; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      a[i][v] = expf(g[i][v]);
      b[i][v] = COMPLEMENT ? -expm1f(g[i][v]) * x[i][v] : x[i][v];
    }
  if (m.first && p.initial_state) {
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      if (m.first >> i & 1) {
        const int n = __shfl_sync(0xffffffffu, m.seq, i);
        const int64_t r = state_row(p, n);
        if (on && r >= 0 && GDR_IN_BOUNDS(n < p.num_seqs && r < p.num_slots && c + V <= p.D)) {
          float h0[V];
          state_load<V>(p.initial_state + r * p.D + c, h0);
#pragma unroll
          for (int v = 0; v < V; ++v) b[i][v] = fmaf(a[i][v], h0[v], b[i][v]);
        }
      }
    }
  }
}

// ---- forward ------------------------------------------------------------
// Reads x and g once and keeps the tokens' a and b in registers while the tile
// waits for what enters it.  STATES_ONLY: the saved chunk states alone.
template <typename IO, int V, bool COMPLEMENT, bool STATES_ONLY>
__global__ void __launch_bounds__(kScanWarps * 32) glr_scan_kernel(GlrArgs p) {
  __shared__ TileShared<V> sh;
  if (bad_offsets(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const Place q = place_of<false>(p, take_tile(p, sh));
  const int64_t t0 = q.tile * kTile + w * kTok;
  const int c = (q.stripe * 32 + lane) * V;
  const bool on = c < p.D;
  float a[kTok][V], b[kTok][V], gs[V], h[V];
  Marks m;
  {
    float x[kTok][V], g[kTok][V];
    load_tokens<IO, V>(p, t0, c, on, x, g);
    m = find_marks(p, t0, lane);
    make_inputs<V, COMPLEMENT>(p, m, c, on, x, g, a, b);
#pragma unroll
    for (int v = 0; v < V; ++v) gs[v] = h[v] = 0.f;
#pragma unroll
    for (int i = 0; i < kTok; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = m.first >> i & 1 ? b[i][v] : fmaf(a[i][v], h[v], b[i][v]);
        gs[v] += g[i][v];
      }
  }
  share_map<V>(sh.G[w], sh.A[w], sh.H[w], lane, gs, h);
  if (lane == 0) sh.closed[w] = m.first != 0;
  __syncthreads();
  Map<V> before = map_before<V, false>(sh, w, lane);
  const bool group_end = q.in_group == p.group - 1;
  if (p.chained && w == kScanWarps - 1 && !group_end) {
    const Map<V> tile = map_before<V, false>(sh, kScanWarps, lane);
    publish_map<V>(p, q, tile, c, on, lane);
  }
  float in[V];
#pragma unroll
  for (int v = 0; v < V; ++v) in[v] = 0.f;
  if (p.chained && !enter_tile<V>(p, sh, q, c, on, w, lane, in)) return;
  if (w == 0 && on && p.chunk_states && GDR_IN_BOUNDS(q.tile < p.tiles && c + V <= p.D))
    row<float, V>::store(p.chunk_states + q.tile * p.D + c, in);
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = before.of(in[v], v);
  if (p.chained && w == kScanWarps - 1 && group_end) {
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      out[v] = sh.closed[w] ? sh.H[w][lane * V + v] : fmaf(sh.A[w][lane * V + v], h[v], sh.H[w][lane * V + v]);
    publish_carry<V>(p, q, out, c, on, lane);
  }
  if (STATES_ONLY) return;
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    const int64_t t = t0 + i;
#pragma unroll
    for (int v = 0; v < V; ++v)
      h[v] = m.first >> i & 1 ? b[i][v] : fmaf(a[i][v], h[v], b[i][v]);
    if (on && t < p.tokens && GDR_IN_BOUNDS(c + V <= p.D))
      row<IO, V>::store(static_cast<IO *>(p.h) + t * p.D + c, h);
    if (p.final_state && (m.last >> i & 1)) {
      const int n = __shfl_sync(0xffffffffu, m.seq, i);
      const int64_t r = state_row(p, n);
      if (on && r >= 0 && GDR_IN_BOUNDS(n < p.num_seqs && r < p.num_slots && c + V <= p.D))
        row<float, V>::store(p.final_state + r * p.D + c, h);
    }
  }
  if (q.tile == 0) pass_empty(p, p.initial_state, p.final_state, true, q.stripe * 32 * V, 32 * V);
}

// ---- backward -----------------------------------------------------------
// The states again from what enters the tile (saved), the gradients from what
// enters it from the tokens after it (chained): x, g and dh are read once.
template <typename IO, int V, bool COMPLEMENT>
__global__ void __launch_bounds__(kScanWarps * 32) glr_gradient_kernel(GlrArgs p) {
  __shared__ TileShared<V> sh;
  __shared__ float state_H[kScanWarps][32 * V];
  __shared__ bool state_closed[kScanWarps];
  if (bad_offsets(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const Place pl = place_of<true>(p, take_tile(p, sh));
  const int64_t t0 = pl.tile * kTile + w * kTok;
  const int c = (pl.stripe * 32 + lane) * V;
  const bool on = c < p.D;
  float x[kTok][V], g[kTok][V], a[kTok][V], b[kTok][V], d[kTok][V];
  load_tokens<IO, V>(p, t0, c, on, x, g);
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
#pragma unroll
    for (int v = 0; v < V; ++v) d[i][v] = 0.f;
    if (on && t0 + i < p.tokens && GDR_IN_BOUNDS(c + V <= p.D))
      row<IO, V>::load(static_cast<const IO *>(p.dh) + (t0 + i) * p.ld_dh + c, d[i]);
  }
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.f;
  if (on && GDR_IN_BOUNDS(pl.tile < p.tiles && c + V <= p.D))
    row<float, V>::load(p.chunk_states + pl.tile * p.D + c, h);
  const Marks m = find_marks(p, t0, lane);
  make_inputs<V, COMPLEMENT>(p, m, c, on, x, g, a, b);
  float gs[V], s[V], q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) gs[v] = s[v] = q[v] = 0.f;
#pragma unroll
  for (int i = 0; i < kTok; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = m.first >> i & 1 ? b[i][v] : fmaf(a[i][v], s[v], b[i][v]);
      gs[v] += g[i][v];
    }
#pragma unroll
  for (int i = kTok - 1; i >= 0; --i) {
    const int n = __shfl_sync(0xffffffffu, m.seq, i);
    const bool last = m.last >> i & 1;  // the gradient of the sequence's final state enters here
    float df[V];
#pragma unroll
    for (int v = 0; v < V; ++v) df[v] = 0.f;
    if (last && p.dfinal && on && GDR_IN_BOUNDS(n < p.num_seqs))
      row<float, V>::load(p.dfinal + (int64_t)n * p.D + c, df);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (last) {
        d[i][v] += df[v];
        q[v] = 0.f;
      }
      q[v] = a[i][v] * (d[i][v] + q[v]);
    }
  }
  share_map<V>(sh.G[w], sh.A[w], sh.H[w], lane, gs, q);
#pragma unroll
  for (int v = 0; v < V; ++v) state_H[w][lane * V + v] = s[v];
  if (lane == 0) {
    sh.closed[w] = m.last != 0;
    state_closed[w] = m.first != 0;
  }
  __syncthreads();
  for (int k = 0; k < w; ++k)  // the state that enters the warp
#pragma unroll
    for (int v = 0; v < V; ++v)
      h[v] = state_closed[k] ? state_H[k][lane * V + v]
                             : fmaf(sh.A[k][lane * V + v], h[v], state_H[k][lane * V + v]);
  Map<V> after = map_before<V, true>(sh, w, lane);
  const bool group_end = pl.in_group == p.group - 1;
  if (p.chained && w == 0 && !group_end) {
    const Map<V> tile = map_before<V, true>(sh, -1, lane);
    publish_map<V>(p, pl, tile, c, on, lane);
  }
  float in[V];
#pragma unroll
  for (int v = 0; v < V; ++v) in[v] = 0.f;
  if (p.chained && !enter_tile<V>(p, sh, pl, c, on, w, lane, in)) return;
#pragma unroll
  for (int v = 0; v < V; ++v) q[v] = after.of(in[v], v);
  if (p.chained && w == 0 && group_end) {
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      out[v] = sh.closed[w] ? sh.H[w][lane * V + v] : fmaf(sh.A[w][lane * V + v], q[v], sh.H[w][lane * V + v]);
    publish_carry<V>(p, pl, out, c, on, lane);
  }
  float before[kTok][V];  // h_{t-1}
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    const bool first = m.first >> i & 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      before[i][v] = first ? 0.f : h[v];
      h[v] = first ? b[i][v] : fmaf(a[i][v], h[v], b[i][v]);
    }
    if (first && p.initial_state) {
      const int n = __shfl_sync(0xffffffffu, m.seq, i);
      if (on && GDR_IN_BOUNDS(n < p.num_seqs))
        state_load<V>(p.initial_state + (int64_t)n * p.D + c, before[i]);
    }
  }
#pragma unroll
  for (int i = kTok - 1; i >= 0; --i) {
    const int64_t t = t0 + i;
    const int n = __shfl_sync(0xffffffffu, m.seq, i);
    float dx[V], dg[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float dt = m.last >> i & 1 ? d[i][v] : d[i][v] + q[v];
      q[v] = a[i][v] * dt;
      dx[v] = COMPLEMENT ? -expm1f(g[i][v]) * dt : dt;
      dg[v] = q[v] * (COMPLEMENT ? before[i][v] - x[i][v] : before[i][v]);
    }
    if (on && t < p.tokens && GDR_IN_BOUNDS(c + V <= p.D)) {
      row<IO, V>::store(static_cast<IO *>(p.dx) + t * p.D + c, dx);
      row<float, V>::store(p.dg + t * p.D + c, dg);
      if (p.dinitial && (m.first >> i & 1) && GDR_IN_BOUNDS(n < p.num_seqs))
        row<float, V>::store(p.dinitial + (int64_t)n * p.D + c, q);
    }
  }
  if (pl.tile == 0) pass_empty(p, p.dfinal, p.dinitial, false, pl.stripe * 32 * V, 32 * V);
}

// Before the chained kernels: zeroes the ticket and the flags, checks the packed
// offsets and writes the status word.
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
    if (threadIdx.x == 0) *p.status = bad ? KDA_DEVICE_BAD_CU_SEQLENS : KDA_DEVICE_OK;
  }
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += (int64_t)gridDim.x * blockDim.x)
    p.ticket[i] = 0;
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
    float x[V], g[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
    if (r >= 0 && GDR_IN_BOUNDS(r < p.num_slots && c + V <= p.D)) {
      row<IO, V>::load(static_cast<const IO *>(p.x) + n * p.ld_x + c, x);
      row<float, V>::load(p.g + n * p.ld_g + c, g);
      state_load<V>(p.final_state + r * p.D + c, h);
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = fmaf(expf(g[v]), h[v], COMPLEMENT ? -expm1f(g[v]) * x[v] : x[v]);
      row<float, V>::store(p.final_state + r * p.D + c, h);
    }
    row<IO, V>::store(static_cast<IO *>(p.h) + (int64_t)n * p.D + c, h);
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
  const int64_t words = p.chained ? 1 + (p.tiles + p.groups) * p.stripes : 0;
  const int64_t want = (words + 1023) / 1024;
  TraceScope tr("glr_begin_kernel", s);
  glr_begin_kernel<<<(unsigned)(want < 1 ? 1 : want > 148 ? 148 : want), 256, 0, s>>>(p, words);
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
  p.group = 4 * kScanWarps;
  p.groups = (p.tiles + p.group - 1) / p.group;
  p.tile_flag = p.ticket + 1;
  p.carry_flag = p.tile_flag + p.tiles * p.stripes;
  return p;
}

template <typename IO, int V, bool COMPLEMENT>
cudaError_t launch_fwd(const GlrArgs &a, cudaStream_t s) {
  const GlrArgs p = with_chain<V>(a);
  cudaError_t e = launch_begin(p, s);
  if (e != cudaSuccess) return e;
  if (p.tiles == 0) return launch_no_tokens(p, false, s);
  TraceScope tr("glr_scan_kernel", s);
  glr_scan_kernel<IO, V, COMPLEMENT, false><<<(unsigned)(p.tiles * p.stripes), kScanWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename IO, int V, bool COMPLEMENT>
cudaError_t launch_bwd(const GlrArgs &a, cudaStream_t s) {
  GlrArgs p = with_chain<V>(a);
  cudaError_t e = launch_begin(p, s);
  if (e != cudaSuccess) return e;
  if (p.tiles == 0) return launch_no_tokens(p, true, s);
  const unsigned grid = (unsigned)(p.tiles * p.stripes);
  if (p.own_chunks) {
    {
      TraceScope tr("glr_scan_kernel", s);
      glr_scan_kernel<IO, V, COMPLEMENT, true><<<grid, kScanWarps * 32, 0, s>>>(p);
    }
    e = launch_begin(p, s);
    if (e != cudaSuccess) return e;
  }
  TraceScope tr("glr_gradient_kernel", s);
  glr_gradient_kernel<IO, V, COMPLEMENT><<<grid, kScanWarps * 32, 0, s>>>(p);
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
