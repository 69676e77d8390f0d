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
    if (on && t < p.tokens) {
      row<IO, V>::load(static_cast<const IO *>(p.x) + t * p.ld_x + c, x[i]);
      row<float, V>::load(p.g + t * p.ld_g + c, g[i]);
    }
  }
}

// The value that enters warp w: what enters the tile, `in`, taken through the
// maps of the warps before it (after it, for REV).
template <int V, bool REV>
__device__ __forceinline__ void enter_warp(const float (&sA)[kScanWarps][32 * V],
                                           const float (&sH)[kScanWarps][32 * V],
                                           const bool (&closed)[kScanWarps], int w, int lane,
                                           float (&h)[V]) {
#pragma unroll
  for (int k = 0; k < kScanWarps; ++k) {
    const int j = REV ? kScanWarps - 1 - k : k;
    if (REV ? j > w : j < w) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = closed[j] ? sH[j][lane * V + v] : fmaf(sA[j][lane * V + v], h[v], sH[j][lane * V + v]);
    }
  }
}

template <int V> struct TileShared {
  float A[kScanWarps][32 * V], H[kScanWarps][32 * V], C[kScanWarps][32 * V];
  bool closed[kScanWarps], closed_rev[kScanWarps];
};

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
        const int64_t r = state_row(p, __shfl_sync(0xffffffffu, m.seq, i));
        if (on && r >= 0) {
          float h0[V];
          state_load<V>(p.initial_state + r * p.D + c, h0);
#pragma unroll
          for (int v = 0; v < V; ++v) b[i][v] = fmaf(a[i][v], h0[v], b[i][v]);
        }
      }
    }
  }
}

// Phase 1: every tile's maps.  FWD: (A, H) of the states; REV: (A, C) of the gradient.
template <typename IO, int V, bool COMPLEMENT, bool REV>
__global__ void __launch_bounds__(kScanWarps * 32) glr_tile_kernel(GlrArgs p) {
  __shared__ TileShared<V> sh;
  if (bad_offsets(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t tile = blockIdx.x, t0 = tile * kTile + w * kTok;
  const int c = (blockIdx.y * 32 + lane) * V;
  const bool on = c < p.D;
  float x[kTok][V], g[kTok][V];
  load_tokens<IO, V>(p, t0, c, on, x, g);
  const Marks m = find_marks(p, t0, lane);
  float gs[V], h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) gs[v] = h[v] = 0.f;
  if (!REV) {
    float a[kTok][V], b[kTok][V];
    make_inputs<V, COMPLEMENT>(p, m, c, on, x, g, a, b);
#pragma unroll
    for (int i = 0; i < kTok; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = m.first >> i & 1 ? b[i][v] : fmaf(a[i][v], h[v], b[i][v]);
        gs[v] += g[i][v];
      }
  } else {
#pragma unroll
    for (int i = kTok - 1; i >= 0; --i) {
      const int64_t t = t0 + i;
      const bool last = m.last >> i & 1;
      const int n = __shfl_sync(0xffffffffu, m.seq, i);
      if (on && t < p.tokens) {
        float d[V];
        row<IO, V>::load(static_cast<const IO *>(p.dh) + t * p.ld_dh + c, d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (last) h[v] = p.dfinal ? __ldg(p.dfinal + (int64_t)n * p.D + c + v) : 0.f;
          h[v] = expf(g[i][v]) * (d[v] + h[v]);
          gs[v] += g[i][v];
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sh.A[w][lane * V + v] = expf(gs[v]);
    sh.H[w][lane * V + v] = h[v];
  }
  if (lane == 0) sh.closed[w] = (REV ? m.last : m.first) != 0;
  // the tile's decay: the sums over its warps
#pragma unroll
  for (int v = 0; v < V; ++v) sh.C[w][lane * V + v] = gs[v];
  __syncthreads();
  if (w != 0) return;
  bool closed = false;
  float hh[V], gt[V];
#pragma unroll
  for (int v = 0; v < V; ++v) hh[v] = gt[v] = 0.f;
  enter_warp<V, REV>(sh.A, sh.H, sh.closed, REV ? -1 : kScanWarps, lane, hh);
#pragma unroll
  for (int k = 0; k < kScanWarps; ++k) {
    closed |= sh.closed[k];
#pragma unroll
    for (int v = 0; v < V; ++v) gt[v] += sh.C[k][lane * V + v];
  }
  if (on)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p.tile_map[(tile * p.D + c + v) * 2] = expf(gt[v]);
      p.tile_map[(tile * p.D + c + v) * 2 + 1] = hh[v];
    }
  if (blockIdx.y == 0 && lane == 0) p.tile_closed[tile] = closed;
}

// Phase 2: what enters each tile, channel by channel.
template <bool REV> __global__ void __launch_bounds__(128) glr_carry_kernel(GlrArgs p) {
  if (bad_offsets(p)) return;
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.D) return;
  float h = 0.f;
  float *out = REV ? p.tile_carry : p.chunk_states;
  for (int64_t k = 0; k < p.tiles; ++k) {
    const int64_t tile = REV ? p.tiles - 1 - k : k;
    out[tile * p.D + c] = h;
    const float2 m = *reinterpret_cast<const float2 *>(p.tile_map + (tile * p.D + c) * 2);
    h = p.tile_closed[tile] ? m.y : fmaf(m.x, h, m.y);
  }
}

// Phase 3, forward: the states of every token.
template <typename IO, int V, bool COMPLEMENT>
__global__ void __launch_bounds__(kScanWarps * 32) glr_apply_kernel(GlrArgs p) {
  __shared__ TileShared<V> sh;
  if (bad_offsets(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t tile = blockIdx.x, t0 = tile * kTile + w * kTok;
  const int c = (blockIdx.y * 32 + lane) * V;
  const bool on = c < p.D;
  float x[kTok][V], g[kTok][V], a[kTok][V], b[kTok][V];
  load_tokens<IO, V>(p, t0, c, on, x, g);
  const Marks m = find_marks(p, t0, lane);
  make_inputs<V, COMPLEMENT>(p, m, c, on, x, g, a, b);
  float gs[V], h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) gs[v] = h[v] = 0.f;
#pragma unroll
  for (int i = 0; i < kTok; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = m.first >> i & 1 ? b[i][v] : fmaf(a[i][v], h[v], b[i][v]);
      gs[v] += g[i][v];
    }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sh.A[w][lane * V + v] = expf(gs[v]);
    sh.H[w][lane * V + v] = h[v];
    h[v] = on ? p.chunk_states[tile * p.D + c + v] : 0.f;
  }
  if (lane == 0) sh.closed[w] = m.first != 0;
  __syncthreads();
  enter_warp<V, false>(sh.A, sh.H, sh.closed, w, lane, h);
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    const int64_t t = t0 + i;
#pragma unroll
    for (int v = 0; v < V; ++v)
      h[v] = m.first >> i & 1 ? b[i][v] : fmaf(a[i][v], h[v], b[i][v]);
    if (on && t < p.tokens && p.h) row<IO, V>::store(static_cast<IO *>(p.h) + t * p.D + c, h);
    if (p.final_state && (m.last >> i & 1)) {
      const int n = __shfl_sync(0xffffffffu, m.seq, i);
      if (on) row<float, V>::store(p.last_state + (int64_t)n * p.D + c, h);
    }
  }
}

// Phase 3, backward: the states again from what enters the tile, then the gradients.
template <typename IO, int V, bool COMPLEMENT>
__global__ void __launch_bounds__(kScanWarps * 32) glr_gradient_kernel(GlrArgs p) {
  __shared__ TileShared<V> sh;
  if (bad_offsets(p)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t tile = blockIdx.x, t0 = tile * kTile + w * kTok;
  const int c = (blockIdx.y * 32 + lane) * V;
  const bool on = c < p.D;
  float x[kTok][V], g[kTok][V], a[kTok][V], b[kTok][V], d[kTok][V];
  load_tokens<IO, V>(p, t0, c, on, x, g);
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
#pragma unroll
    for (int v = 0; v < V; ++v) d[i][v] = 0.f;
    if (on && t0 + i < p.tokens)
      row<IO, V>::load(static_cast<const IO *>(p.dh) + (t0 + i) * p.ld_dh + c, d[i]);
  }
  const Marks m = find_marks(p, t0, lane);
  make_inputs<V, COMPLEMENT>(p, m, c, on, x, g, a, b);
  float gs[V], h[V], q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) gs[v] = h[v] = q[v] = 0.f;
#pragma unroll
  for (int i = 0; i < kTok; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = m.first >> i & 1 ? b[i][v] : fmaf(a[i][v], h[v], b[i][v]);
      gs[v] += g[i][v];
    }
#pragma unroll
  for (int i = kTok - 1; i >= 0; --i) {
    const int n = __shfl_sync(0xffffffffu, m.seq, i);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (m.last >> i & 1) {  // the gradient of the sequence's final state enters here
        d[i][v] += on && p.dfinal ? __ldg(p.dfinal + (int64_t)n * p.D + c + v) : 0.f;
        q[v] = 0.f;
      }
      q[v] = a[i][v] * (d[i][v] + q[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sh.A[w][lane * V + v] = expf(gs[v]);
    sh.H[w][lane * V + v] = h[v];
    sh.C[w][lane * V + v] = q[v];
    h[v] = on ? p.chunk_states[tile * p.D + c + v] : 0.f;
    q[v] = on ? p.tile_carry[tile * p.D + c + v] : 0.f;
  }
  if (lane == 0) {
    sh.closed[w] = m.first != 0;
    sh.closed_rev[w] = m.last != 0;
  }
  __syncthreads();
  enter_warp<V, false>(sh.A, sh.H, sh.closed, w, lane, h);
  enter_warp<V, true>(sh.A, sh.C, sh.closed_rev, w, lane, q);
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
      const int64_t r = state_row(p, __shfl_sync(0xffffffffu, m.seq, i));
      if (on && r >= 0) state_load<V>(p.initial_state + r * p.D + c, before[i]);
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
    if (on && t < p.tokens) {
      row<IO, V>::store(static_cast<IO *>(p.dx) + t * p.D + c, dx);
      row<float, V>::store(p.dg + t * p.D + c, dg);
      if (p.dinitial && (m.first >> i & 1)) row<float, V>::store(p.dinitial + (int64_t)n * p.D + c, q);
    }
  }
}

// The states that leave the sequences: of those without tokens what enters
// them.  (Final states wait for this launch in the workspace: they may go to
// the very slots that the initial states are read from.)
__global__ void __launch_bounds__(256) glr_finish_kernel(GlrArgs p, bool backward) {
  if (bad_offsets(p)) return;
  const int n = blockIdx.x;
  const bool empty = p.cu_seqlens ? __ldg(p.cu_seqlens + n) == __ldg(p.cu_seqlens + n + 1) : p.T == 0;
  if (backward && !empty) return;
  const int64_t r = backward ? n : state_row(p, n);
  if (r < 0) return;
  const float *src = backward ? p.dfinal : p.initial_state;
  float *dst = backward ? p.dinitial : p.final_state;
  for (int c = threadIdx.x; c < p.D; c += blockDim.x)
    dst[r * p.D + c] = !empty ? p.last_state[(int64_t)n * p.D + c] : src ? src[r * p.D + c] : 0.f;
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
    if (r >= 0) {
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

template <typename IO, int V, bool COMPLEMENT>
cudaError_t launch_chunk_states(const GlrArgs &p, cudaStream_t s) {
  const dim3 grid((unsigned)p.tiles, (unsigned)((p.D + 32 * V - 1) / (32 * V)));
  if (p.tiles == 0) return cudaSuccess;
  {
    TraceScope tr("glr_tile_kernel", s);
    glr_tile_kernel<IO, V, COMPLEMENT, false><<<grid, kScanWarps * 32, 0, s>>>(p);
  }
  TraceScope tr("glr_carry_kernel", s);
  glr_carry_kernel<false><<<(p.D + 127) / 128, 128, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename IO, int V, bool COMPLEMENT>
cudaError_t launch_fwd(const GlrArgs &p, cudaStream_t s) {
  const dim3 grid((unsigned)p.tiles, (unsigned)((p.D + 32 * V - 1) / (32 * V)));
  if (p.tiles > 0) {
    launch_chunk_states<IO, V, COMPLEMENT>(p, s);
    TraceScope tr("glr_apply_kernel", s);
    glr_apply_kernel<IO, V, COMPLEMENT><<<grid, kScanWarps * 32, 0, s>>>(p);
  }
  if (p.num_seqs > 0 && p.final_state) {
    TraceScope tr("glr_finish_kernel", s);
    glr_finish_kernel<<<p.num_seqs, 256, 0, s>>>(p, false);
  }
  return cudaGetLastError();
}

template <typename IO, int V, bool COMPLEMENT>
cudaError_t launch_bwd(const GlrArgs &p, cudaStream_t s) {
  const dim3 grid((unsigned)p.tiles, (unsigned)((p.D + 32 * V - 1) / (32 * V)));
  if (p.tiles > 0) {
    {
      TraceScope tr("glr_tile_kernel", s);
      glr_tile_kernel<IO, V, COMPLEMENT, true><<<grid, kScanWarps * 32, 0, s>>>(p);
    }
    {
      TraceScope tr("glr_carry_kernel", s);
      glr_carry_kernel<true><<<(p.D + 127) / 128, 128, 0, s>>>(p);
    }
    TraceScope tr("glr_gradient_kernel", s);
    glr_gradient_kernel<IO, V, COMPLEMENT><<<grid, kScanWarps * 32, 0, s>>>(p);
  }
  if ((p.cu_seqlens || p.T == 0) && p.num_seqs > 0 && p.dinitial) {
    TraceScope tr("glr_finish_kernel", s);
    glr_finish_kernel<<<p.num_seqs, 256, 0, s>>>(p, true);
  }
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
cudaError_t launch_glr_chunk_states(const GlrArgs &p, cudaStream_t s) {
  GDR_GLR_DISPATCH(launch_chunk_states);
}
cudaError_t launch_glr_bwd(const GlrArgs &p, cudaStream_t s) { GDR_GLR_DISPATCH(launch_bwd); }
cudaError_t launch_glr_step(const GlrArgs &p, cudaStream_t s) { GDR_GLR_DISPATCH(launch_step); }

}  // namespace gdr
