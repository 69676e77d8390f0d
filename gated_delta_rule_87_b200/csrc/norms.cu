// RMS norms on both sides of a mixer block, forward and backward (sm_100a).
//
// Gated norm, per head row x of d channels, with weight w and gate z:
//     u = x r,  r = 1 / sqrt(mean(x^2) + eps),   y = u w s(z),  s = z sigmoid(z) | sigmoid(z) | 1
//     du = dy w s,  dx = r (du - u mean(du u)),  dz = dy u w s'(z),  dw = sum over rows of dy u s
// Residual add and norm:
//     t = residual + scale y,  n = t r w
//     d = dt + r (dn w - u mean(dn w u)),  dresidual = d,  dy = scale d,
//     dw = sum of dn u,  dscale = sum of d y
//
// Every row is read once, held in registers and each output written once: the
// kernels are bound by HBM.  mean(du u) = r mean(du x), so the backward pass
// takes both of its row sums in one reduction.  A row belongs to a group of
// threads: 8, 16 or 32 lanes of a warp for short rows, a whole block for longer
// ones; the next row's loads are under way while this one is worked on.
//
// Accesses are 16 bytes wide on 16-byte boundaries of the whole tensor, whatever
// the row length: a row that begins `shift` elements past a boundary is cut there
// (its first and last pieces are then partial, element by element).  A group's
// rows are a multiple of 8 rows apart, so its shift, and with it the columns of
// each thread, stay the same: the column sums of the weights' gradients are held
// in registers, then summed over a block's groups and over the blocks in a fixed
// order (no atomics: the same inputs give the same bits).
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace gdr {
namespace {

constexpr int kBlockThreads = 640;  // most threads of a block that shares one row
constexpr int kCachedDevices = 64;

// V elements as they are stored: V sizeof(T) bytes in 16-byte pieces, or one element.
template <typename T, int V> struct Pack {
  static constexpr int N = V * (int)sizeof(T) / 16;
  uint4 q[N];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4 &u = q[i / 4];
    return i % 4 == 0 ? u.x : i % 4 == 1 ? u.y : i % 4 == 2 ? u.z : u.w;
  }
  __device__ __forceinline__ float at(int v) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(word(v));
    else return v & 1 ? bf16_hi(word(v / 2)) : bf16_lo(word(v / 2));
  }
  // `whole`: all V elements are the row's, else those with 0 <= c + v < d
  // (plain loads: some callers write the tensor that they read, row by row)
  __device__ __forceinline__ void load(const T *row, int c, int d, bool whole) {
    const T *p = row + c;
    if (whole) {
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = reinterpret_cast<const uint4 *>(p)[i];
    } else {
      uint32_t w[4 * N];
#pragma unroll
      for (int i = 0; i < 4 * N; ++i) w[i] = 0;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (c + v >= 0 && c + v < d) {
          if constexpr (sizeof(T) == 4) w[v] = reinterpret_cast<const uint32_t *>(p)[v];
          else w[v / 2] |= (uint32_t)reinterpret_cast<const unsigned short *>(p)[v] << 16 * (v & 1);
        }
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
};
template <typename T> struct Pack<T, 1> {
  T r;
  __device__ __forceinline__ void zero() { r = T(0.f); }
  __device__ __forceinline__ float at(int) const { return float(r); }
  __device__ __forceinline__ void load(const T *row, int c, int, bool) { r = row[c]; }
};
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *row, int c, int d, bool whole, const float (&x)[V]) {
  T *p = row + c;
  if constexpr (V == 1) {
    io<T>::store(p, x[0]);
  } else if (whole) {
    uint32_t w[V * sizeof(T) / 4];
#pragma unroll
    for (int i = 0; i < (int)(V * sizeof(T) / 4); ++i)
      w[i] = sizeof(T) == 4 ? __float_as_uint(x[i]) : pack_bf16x2(x[2 * i % V], x[(2 * i + 1) % V]);  // (% V: the unused arm)
#pragma unroll
    for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i)
      reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c + v >= 0 && c + v < d) io<T>::store(p + v, x[v]);
  }
}

// A group of threads that shares one row: LANES lanes of a warp, or the block
// (LANES = 0); and its walk over the rows.
template <int V, int NV, int LANES> struct Group {
  int lane, index, per_block, size, d;
  int64_t row, step, rows;
  int c[NV];  // first column of each of the thread's pieces, and what they are
  bool any[NV], whole[NV];
  float2 *buf;  // [2][32] shared, block groups only
  int turn;
  __device__ __forceinline__ Group(float2 *shared, int64_t rows_, int d_) : d(d_), rows(rows_), buf(shared), turn(0) {
    if (LANES) {
      lane = threadIdx.x % LANES;
      index = threadIdx.x / LANES;
      per_block = blockDim.x / LANES;
      size = LANES;
    } else {
      lane = threadIdx.x;
      index = 0;
      per_block = 1;
      size = blockDim.x;
    }
    row = (int64_t)blockIdx.x * per_block + index;
    step = (int64_t)gridDim.x * per_block;
    const int shift = (int)((row % V) * (d % V) % V);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      c[i] = (i * size + lane) * V - shift;
      any[i] = c[i] < d;
      whole[i] = c[i] >= 0 && c[i] + V <= d;
    }
  }
  // rows that the block walks: every group takes part in every step's sums
  __device__ __forceinline__ bool more(int64_t r) const { return r - index < rows; }
  __device__ __forceinline__ bool in(int i, int v) const { return c[i] + v >= 0 && c[i] + v < d; }
  // Sums over the group, the same bits in each of its threads.  Every thread of
  // the block calls it as often as every other.
  __device__ __forceinline__ float2 sum(float a, float b) {
#pragma unroll
    for (int o = (LANES ? LANES : 32) / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (LANES) return make_float2(a, b);
    const int w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float2 *s = buf + 32 * turn;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[w] = make_float2(a, b);
    __syncthreads();
    const int l = threadIdx.x & 31;
    float2 t = l < warps ? s[l] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
      t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
    }
    return t;
  }
};

// A thread's columns of a [d] vector (ones where there is none), the same for
// every row: in registers for the lanes of a warp, in a shared-memory slot of the
// thread's own for a block (no barrier: nobody else reads it).
template <int V, int NV, int LANES> struct Columns {
  float r[LANES ? NV : 1][V];
  float *slot;
  __device__ __forceinline__ Columns(const Group<V, NV, LANES> &grp, const float *p, float *shared) {
    slot = shared + threadIdx.x * V;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float x[V];
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = p && grp.in(i, v) ? __ldg(p + grp.c[i] + v) : 1.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (LANES) r[LANES ? i : 0][v] = x[v];
        else slot[(size_t)i * blockDim.x * V + v] = x[v];
      }
    }
  }
  __device__ __forceinline__ void get(int i, float (&x)[V]) const {
    if (LANES) {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = r[LANES ? i : 0][v];
    } else if constexpr (V == 1) {
      x[0] = slot[(size_t)i * blockDim.x];
    } else {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(slot + (size_t)i * blockDim.x * V + v);
        x[v] = f.x; x[v + 1] = f.y; x[v + 2] = f.z; x[v + 3] = f.w;
      }
    }
  }
};
// shared memory of one such vector in a block
template <int V, int NV, int LANES> __device__ __forceinline__ float *column_slots(float *shared, int k) {
  return LANES ? shared : shared + (size_t)k * NV * blockDim.x * V;
}

// sigmoid.  bf16 results keep 8 bits, so the intrinsics' few ulp are far below
// their rounding; fp32 ones take the accurate functions.
template <typename IO> __device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(IO) == 2) return __fdividef(1.f, 1.f + __expf(-z));
  else return 1.f / (1.f + expf(-z));
}
// the gate's value, and its slope, from z and g = sigmoid(z)
template <int GATE> __device__ __forceinline__ float gate_value(float z, float g) {
  return GATE == KDA_GATE_NONE ? 1.f : GATE == KDA_GATE_SILU ? z * g : g;
}
template <int GATE> __device__ __forceinline__ float gate_slope(float z, float g) {
  return GATE == KDA_GATE_SILU ? g * (1.f + z * (1.f - g)) : g * (1.f - g);
}

// Where a row of a [tokens, H, d] tensor begins, tokens ld elements apart.
struct HeadRow {
  int64_t tok;
  int head;
  __device__ __forceinline__ HeadRow(int64_t row, int H) : tok(row / H), head((int)(row - tok * H)) {}
  __device__ __forceinline__ int64_t at(int64_t ld, int d) const { return tok * ld + (int64_t)head * d; }
};

template <typename IO, int V, int NV, int LANES, int GATE>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads) gated_norm_fwd_kernel(GatedNormArgs p) {
  __shared__ float2 buf[64];
  extern __shared__ __align__(16) float shared[];
  Group<V, NV, LANES> grp(buf, p.tokens * p.H, p.d);
  const Columns<V, NV, LANES> weight(grp, p.weight, shared);
  Pack<IO, V> x[NV], z[NV];
  auto load = [&](int64_t row) {
    if (row >= grp.rows) return;
    const HeadRow at(row, p.H);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i].zero();
      z[i].zero();
      if (!grp.any[i] || !GDR_IN_BOUNDS(at.tok < p.tokens)) continue;
      x[i].load(static_cast<const IO *>(p.x) + at.at(p.ld_x, p.d), grp.c[i], p.d, grp.whole[i]);
      if (GATE != KDA_GATE_NONE)
        z[i].load(static_cast<const IO *>(p.z) + at.at(p.ld_z, p.d), grp.c[i], p.d, grp.whole[i]);
    }
  };
  load(grp.row);
  for (int64_t row = grp.row; grp.more(row); row += grp.step) {
    float xv[NV][V], sv[NV][V], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        xv[i][v] = x[i].at(v);
        const float zv = z[i].at(v);
        sv[i][v] = GATE == KDA_GATE_NONE ? 1.f : gate_value<GATE>(zv, sigmoid<IO>(zv));
        ss = fmaf(xv[i][v], xv[i][v], ss);
      }
    load(row + grp.step);
    const float inv = rsqrtf(grp.sum(ss, 0.f).x / (float)p.d + p.eps);
    if (row >= grp.rows) continue;
    IO *y = static_cast<IO *>(p.y) + row * p.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[V];
      weight.get(i, w);
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] *= xv[i][v] * inv * sv[i][v];
      if (grp.any[i] && GDR_IN_BOUNDS(row < grp.rows)) store_vec<IO, V>(y, grp.c[i], p.d, grp.whole[i], w);
    }
  }
}

// Sums acc over the block's groups and writes the block's row of partial sums.
template <int V, int NV, int LANES>
__device__ __forceinline__ void write_partial(const Group<V, NV, LANES> &grp, const float (&acc)[NV][V],
                                              float *smem, float *partial) {
  const int d = grp.d;
  float *to = LANES ? smem + grp.index * d : partial + (int64_t)blockIdx.x * d;
  if (LANES) __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (grp.in(i, v) && GDR_IN_BOUNDS(blockIdx.x < kNormBlocks)) to[grp.c[i] + v] = acc[i][v];
  if (!LANES) return;
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float t = 0.f;
    for (int k = 0; k < grp.per_block; ++k) t += smem[k * d + c];
    if (GDR_IN_BOUNDS(blockIdx.x < kNormBlocks)) partial[(int64_t)blockIdx.x * d + c] = t;
  }
}

template <typename IO, int V, int NV, int LANES, int GATE>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads, LANES ? 3 : 1)
gated_norm_bwd_kernel(GatedNormArgs p) {
  __shared__ float2 buf[64];
  extern __shared__ __align__(16) float shared[];
  Group<V, NV, LANES> grp(buf, p.tokens * p.H, p.d);
  constexpr bool EARLY = NV == 1;  // the next row's loads under way
  const Columns<V, NV, LANES> weight(grp, p.weight, shared);
  float acc[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) acc[i][v] = 0.f;
  Pack<IO, V> dy[NV], x[NV], z[NV];
  auto load = [&](int64_t row) {
    if (row >= grp.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[i].zero();
        dy[i].zero();
        z[i].zero();
      }
      return;
    }
    const HeadRow at(row, p.H);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i].zero();
      dy[i].zero();
      z[i].zero();
      if (!grp.any[i] || !GDR_IN_BOUNDS(at.tok < p.tokens)) continue;
      x[i].load(static_cast<const IO *>(p.x) + at.at(p.ld_x, p.d), grp.c[i], p.d, grp.whole[i]);
      dy[i].load(static_cast<const IO *>(p.dy) + at.at(p.ld_dy, p.d), grp.c[i], p.d, grp.whole[i]);
      if (GATE != KDA_GATE_NONE)
        z[i].load(static_cast<const IO *>(p.z) + at.at(p.ld_z, p.d), grp.c[i], p.d, grp.whole[i]);
    }
  };
  load(grp.row);
  for (int64_t row = grp.row; grp.more(row); row += grp.step) {
    // xv: x; sv: the gate's value; gv: dy; zv: its slope
    float xv[NV][V], sv[NV][V], gv[NV][V], zv[NV][V], ss = 0.f, sd = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[V];
      weight.get(i, w);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        xv[i][v] = x[i].at(v);
        gv[i][v] = dy[i].at(v);
        sv[i][v] = 1.f;
        zv[i][v] = 0.f;
        if (GATE != KDA_GATE_NONE) {
          const float zz = z[i].at(v), g = sigmoid<IO>(zz);
          sv[i][v] = gate_value<GATE>(zz, g);
          zv[i][v] = gate_slope<GATE>(zz, g);
        }
        ss = fmaf(xv[i][v], xv[i][v], ss);
        sd = fmaf(gv[i][v] * w[v] * sv[i][v], xv[i][v], sd);
      }
    }
    if (EARLY) load(row + grp.step);
    const float2 t = grp.sum(ss, sd);
    const float inv = rsqrtf(t.x / (float)p.d + p.eps);
    const float m = inv * inv * (t.y / (float)p.d);  // mean(du u) r
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float dx[V], dz[V], w[V];
      weight.get(i, w);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float gu = gv[i][v] * (xv[i][v] * inv);
        dx[v] = inv * (gv[i][v] * w[v] * sv[i][v] - xv[i][v] * m);
        dz[v] = gu * w[v] * zv[i][v];
        acc[i][v] = fmaf(gu, sv[i][v], acc[i][v]);
      }
      if (row < grp.rows && grp.any[i] && GDR_IN_BOUNDS(row < grp.rows)) {
        store_vec<IO, V>(static_cast<IO *>(p.dx) + row * p.d, grp.c[i], p.d, grp.whole[i], dx);
        if (GATE != KDA_GATE_NONE)
          store_vec<IO, V>(static_cast<IO *>(p.dz) + row * p.d, grp.c[i], p.d, grp.whole[i], dz);
      }
    }
    if (!EARLY) load(row + grp.step);
  }
  if (p.partial) write_partial(grp, acc, shared, p.partial);
}

template <typename RES, typename IO, int V, int NV, int LANES>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads) add_norm_fwd_kernel(AddNormArgs p) {
  __shared__ float2 buf[64];
  extern __shared__ __align__(16) float shared[];
  Group<V, NV, LANES> grp(buf, p.rows, p.D);
  const Columns<V, NV, LANES> weight(grp, p.weight, column_slots<V, NV, LANES>(shared, 0));
  const Columns<V, NV, LANES> scale(grp, p.scale, column_slots<V, NV, LANES>(shared, 1));
  Pack<RES, V> r[NV];
  Pack<IO, V> y[NV];
  auto load = [&](int64_t row) {
    if (row >= grp.rows) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      r[i].zero();
      y[i].zero();
      if (!grp.any[i] || !GDR_IN_BOUNDS(row < p.rows)) continue;
      r[i].load(static_cast<const RES *>(p.residual) + row * p.D, grp.c[i], p.D, grp.whole[i]);
      y[i].load(static_cast<const IO *>(p.y) + row * p.D, grp.c[i], p.D, grp.whole[i]);
    }
  };
  load(grp.row);
  for (int64_t row = grp.row; grp.more(row); row += grp.step) {
    float t[NV][V], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float sc[V];
      scale.get(i, sc);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        t[i][v] = fmaf(sc[v], y[i].at(v), r[i].at(v));
        ss = fmaf(t[i][v], t[i][v], ss);
      }
      if (row < grp.rows && grp.any[i] && GDR_IN_BOUNDS(row < p.rows))
        store_vec<RES, V>(static_cast<RES *>(p.residual_out) + row * p.D, grp.c[i], p.D, grp.whole[i], t[i]);
    }
    load(row + grp.step);
    const float inv = rsqrtf(grp.sum(ss, 0.f).x / (float)p.D + p.eps);
    if (row >= grp.rows) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[V];
      weight.get(i, w);
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] *= t[i][v] * inv;
      if (grp.any[i] && GDR_IN_BOUNDS(row < p.rows))
        store_vec<IO, V>(static_cast<IO *>(p.n) + row * p.D, grp.c[i], p.D, grp.whole[i], w);
    }
  }
}

template <typename RES, typename IO, int V, int NV, int LANES>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads) add_norm_bwd_kernel(AddNormArgs p) {
  __shared__ float2 buf[64];
  extern __shared__ __align__(16) float shared[];
  Group<V, NV, LANES> grp(buf, p.rows, p.D);
  constexpr bool EARLY = NV == 1;  // the next row's loads under way
  const bool want_dscale = p.dscale != nullptr;
  const Columns<V, NV, LANES> weight(grp, p.weight, column_slots<V, NV, LANES>(shared, 0));
  const Columns<V, NV, LANES> scale(grp, p.scale, column_slots<V, NV, LANES>(shared, 1));
  float aw[NV][V], as[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) aw[i][v] = as[i][v] = 0.f;
  Pack<RES, V> t[NV], dt[NV];
  Pack<IO, V> dn[NV], y[NV];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      t[i].zero();
      dt[i].zero();
      dn[i].zero();
      y[i].zero();
      if (row >= grp.rows || !grp.any[i] || !GDR_IN_BOUNDS(row < p.rows)) continue;
      t[i].load(static_cast<const RES *>(p.residual_out) + row * p.D, grp.c[i], p.D, grp.whole[i]);
      dn[i].load(static_cast<const IO *>(p.dn) + row * p.D, grp.c[i], p.D, grp.whole[i]);
      if (p.dresidual_out)
        dt[i].load(static_cast<const RES *>(p.dresidual_out) + row * p.D, grp.c[i], p.D, grp.whole[i]);
      if (want_dscale) y[i].load(static_cast<const IO *>(p.y) + row * p.D, grp.c[i], p.D, grp.whole[i]);
    }
  };
  load(grp.row);
  for (int64_t row = grp.row; grp.more(row); row += grp.step) {
    Pack<RES, V> ct[NV], cdt[NV];
    Pack<IO, V> cdn[NV], cy[NV];
    float ss = 0.f, sd = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[V];
      weight.get(i, w);
      ct[i] = t[i];
      cdt[i] = dt[i];
      cdn[i] = dn[i];
      cy[i] = y[i];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        ss = fmaf(ct[i].at(v), ct[i].at(v), ss);
        sd = fmaf(cdn[i].at(v) * w[v], ct[i].at(v), sd);
      }
    }
    if (EARLY) load(row + grp.step);
    const float2 s = grp.sum(ss, sd);
    const float inv = rsqrtf(s.x / (float)p.D + p.eps);
    const float m = inv * inv * (s.y / (float)p.D);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float d[V], dy[V], w[V], sc[V];
      weight.get(i, w);
      scale.get(i, sc);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float tv = ct[i].at(v), gv = cdn[i].at(v);
        d[v] = cdt[i].at(v) + inv * (gv * w[v] - tv * m);
        aw[i][v] = fmaf(gv, tv * inv, aw[i][v]);
        as[i][v] = fmaf(d[v], cy[i].at(v), as[i][v]);
        dy[v] = d[v] * sc[v];
      }
      if (row < grp.rows && grp.any[i] && GDR_IN_BOUNDS(row < p.rows)) {
        store_vec<RES, V>(static_cast<RES *>(p.dresidual) + row * p.D, grp.c[i], p.D, grp.whole[i], d);
        if (p.dy) store_vec<IO, V>(static_cast<IO *>(p.dy) + row * p.D, grp.c[i], p.D, grp.whole[i], dy);
      }
    }
    if (!EARLY) load(row + grp.step);
  }
  if (p.dweight) write_partial(grp, aw, shared, p.partial);
  if (want_dscale) write_partial(grp, as, shared, p.partial + (int64_t)kNormBlocks * p.D);
}

// out[c] = sum of partial[b][c] over the blocks, in a fixed order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *__restrict__ partial0,
                                                          float *out0, const float *partial1,
                                                          float *out1, int blocks, int d) {
  const float *partial = blockIdx.y ? partial1 : partial0;
  float *out = blockIdx.y ? out1 : out0;
  if (!out) return;
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float t = 0.f;
  if (c < d)
    for (int b = threadIdx.y; b < blocks; b += 32) t += partial[(int64_t)b * d + c];
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  t = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int co = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && co < d) out[co] = t;
}

struct Plan {
  int lanes, nv, threads;  // lanes 0: a block a row
  size_t smem;             // the columns of `vectors` vectors (a block), or the groups' column sums
};
// Rows of up to 32 pieces go to the 8, 16 or 32 lanes of a warp that hold one
// piece each, longer ones to a block with one piece a thread, up to 640
// threads, and more pieces a thread only beyond that.
Plan plan(int d, int V, bool backward, int vectors) {
  Plan q{};
  const int vecs = d % V == 0 ? d / V : (d + 2 * V - 2) / V;  // pieces of a row that begins anywhere
  q.nv = 1;
  if (vecs <= 32) {
    q.lanes = vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32;
    q.threads = 256;
    q.smem = backward ? (size_t)(q.threads / q.lanes) * d * sizeof(float) : 0;
  } else {
    while ((vecs + q.nv - 1) / q.nv > kBlockThreads) q.nv *= 2;
    q.threads = ((vecs + q.nv - 1) / q.nv + 31) / 32 * 32;
    q.smem = (size_t)vectors * q.nv * q.threads * V * sizeof(float);
  }
  return q;
}

// Two vectors of the longest row, its pieces shared out over whole warps, take at
// most 2 (kNormMaxRow + 32 x 32) floats.
constexpr int kMostShared = 2 * (kNormMaxRow + 32 * 32) * (int)sizeof(float);

// Blocks that run at once on the current device for this kernel and plan: a
// whole number of them walks the rows (asked once a device and block size).
template <auto KERNEL> cudaError_t resident_blocks(const Plan &q, int *blocks) {
  static std::atomic<int> cache[kCachedDevices][kBlockThreads / 32 + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int> *slot = dev >= 0 && dev < kCachedDevices ? &cache[dev][q.threads / 32] : nullptr;
  *blocks = slot ? slot->load(std::memory_order_relaxed) : 0;
  if (*blocks > 0) return cudaSuccess;
  int per_sm = 0;
  if (q.smem > 48 * 1024) e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERNEL, q.threads, q.smem);
  if (e != cudaSuccess) return e;
  *blocks = sm_count() * (per_sm > 0 ? per_sm : 1);
  if (slot) slot->store(*blocks, std::memory_order_relaxed);
  return cudaSuccess;
}

// Launches a norm kernel over `rows` rows; `blocks` becomes its grid.  A group's
// rows are `blocks` times its block's groups apart: a multiple of 8 where the
// rows' shifts differ and a group has more than one.
template <auto KERNEL, typename ARGS>
cudaError_t launch_rows(const char *name, const ARGS &p, const Plan &q, int64_t rows, cudaStream_t s, int *blocks) {
  int most = 0;
  cudaError_t e = resident_blocks<KERNEL>(q, &most);
  if (e != cudaSuccess) return e;
  if (most > kNormBlocks) most = kNormBlocks;
  if (most >= 8) most -= most % 8;
  const int per = q.lanes ? q.threads / q.lanes : 1;
  const int64_t want = (rows + per - 1) / per;
  *blocks = (int)(want < most ? want : most);
  TraceScope tr(name, s);
  KERNEL<<<*blocks, q.threads, q.smem, s>>>(p);
  return cudaGetLastError();
}
static_assert(kNormBlocks % 8 == 0, "a full grid keeps the groups' shifts");

template <typename T> cudaError_t sum_columns(const T &p, float *out0, float *out1, int d, int blocks, cudaStream_t s) {
  if (!out0 && !out1) return cudaSuccess;
  TraceScope tr("column_sum_kernel", s);
  column_sum_kernel<<<dim3((d + 31) / 32, out1 ? 2 : 1), dim3(32, 32), 0, s>>>(
      p.partial, out0, p.partial + (int64_t)kNormBlocks * d, out1, blocks, d);
  return cudaGetLastError();
}

// LAUNCH(pieces a thread, lanes) of a plan
#define GDR_NORM_PLAN(q, LAUNCH)                    \
  do {                                              \
    if (q.lanes == 8) LAUNCH(1, 8);                 \
    else if (q.lanes == 16) LAUNCH(1, 16);          \
    else if (q.lanes == 32) LAUNCH(1, 32);          \
    else if (q.nv == 1) LAUNCH(1, 0);               \
    else if (q.nv == 2) LAUNCH(2, 0);               \
    else if (q.nv == 4) LAUNCH(4, 0);               \
    else if (q.nv == 8) LAUNCH(8, 0);               \
    else if constexpr (V < 8) {                     \
      if (q.nv == 16) LAUNCH(16, 0);                \
      else if constexpr (V == 1) LAUNCH(32, 0);     \
    }                                               \
  } while (0)
static_assert(kNormMaxRow + 8 <= kBlockThreads * 8 * 8 && kNormMaxRow + 4 <= kBlockThreads * 4 * 16 &&
                  kNormMaxRow <= kBlockThreads * 32,
              "a block holds the longest row");

template <typename IO, int V, int GATE>
cudaError_t gated_gate(const GatedNormArgs &p, bool back, cudaStream_t s) {
  const Plan q = plan(p.d, V, back, 1);
  const int64_t rows = p.tokens * p.H;
  int blocks = 0;
  cudaError_t e = cudaErrorInvalidValue;
  if (!back) {
#define GDR_LAUNCH(NV, LANES) \
  e = launch_rows<gated_norm_fwd_kernel<IO, V, NV, LANES, GATE>>("gated_norm_fwd_kernel", p, q, rows, s, &blocks)
    GDR_NORM_PLAN(q, GDR_LAUNCH);
#undef GDR_LAUNCH
    return e;
  }
#define GDR_LAUNCH(NV, LANES) \
  e = launch_rows<gated_norm_bwd_kernel<IO, V, NV, LANES, GATE>>("gated_norm_bwd_kernel", p, q, rows, s, &blocks)
  GDR_NORM_PLAN(q, GDR_LAUNCH);
#undef GDR_LAUNCH
  return e == cudaSuccess ? sum_columns(p, p.dweight, nullptr, p.d, blocks, s) : e;
}

template <typename IO, int V> cudaError_t gated_vec(const GatedNormArgs &p, bool back, cudaStream_t s) {
  switch (p.gate) {
    case KDA_GATE_SILU: return gated_gate<IO, V, KDA_GATE_SILU>(p, back, s);
    case KDA_GATE_SIGMOID: return gated_gate<IO, V, KDA_GATE_SIGMOID>(p, back, s);
    default: return gated_gate<IO, V, KDA_GATE_NONE>(p, back, s);
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 16-byte accesses where every tensor begins on 16 bytes, and either its rows do
// too or its tokens follow each other without a gap.
template <typename IO> cudaError_t gated_io(const GatedNormArgs &p, bool back, cudaStream_t s) {
  constexpr int V = 16 / sizeof(IO);
  const int64_t row = (int64_t)p.H * p.d;
  const bool packed = p.ld_x == row && (!p.z || p.ld_z == row) && (!p.dy || p.ld_dy == row);
  const bool even = p.d % V == 0 && p.ld_x % V == 0 && p.ld_z % V == 0 && p.ld_dy % V == 0;
  const bool wide = (packed || even) && aligned16(p.x) && aligned16(p.z) && aligned16(p.y) && aligned16(p.dy) &&
                    aligned16(p.dx) && aligned16(p.dz);
  return wide ? gated_vec<IO, V>(p, back, s) : gated_vec<IO, 1>(p, back, s);
}

template <typename RES, typename IO, int V>
cudaError_t add_vec(const AddNormArgs &p, bool back, cudaStream_t s) {
  const Plan q = plan(p.D, V, back, 2);
  int blocks = 0;
  cudaError_t e = cudaErrorInvalidValue;
  if (!back) {
#define GDR_LAUNCH(NV, LANES) \
  e = launch_rows<add_norm_fwd_kernel<RES, IO, V, NV, LANES>>("add_norm_fwd_kernel", p, q, p.rows, s, &blocks)
    GDR_NORM_PLAN(q, GDR_LAUNCH);
#undef GDR_LAUNCH
    return e;
  }
#define GDR_LAUNCH(NV, LANES) \
  e = launch_rows<add_norm_bwd_kernel<RES, IO, V, NV, LANES>>("add_norm_bwd_kernel", p, q, p.rows, s, &blocks)
  GDR_NORM_PLAN(q, GDR_LAUNCH);
#undef GDR_LAUNCH
  return e == cudaSuccess ? sum_columns(p, p.dweight, p.dscale, p.D, blocks, s) : e;
}

template <typename RES, typename IO> cudaError_t add_io(const AddNormArgs &p, bool back, cudaStream_t s) {
  constexpr int V = 16 / sizeof(IO);
  const bool wide = aligned16(p.residual) && aligned16(p.y) && aligned16(p.residual_out) && aligned16(p.n) &&
                    aligned16(p.dn) && aligned16(p.dresidual_out) && aligned16(p.dresidual) && aligned16(p.dy);
  return wide ? add_vec<RES, IO, V>(p, back, s) : add_vec<RES, IO, 1>(p, back, s);
}

cudaError_t add_any(const AddNormArgs &p, bool back, cudaStream_t s) {
  if (!p.bf16) return add_io<float, float>(p, back, s);
  return p.res_bf16 ? add_io<__nv_bfloat16, __nv_bfloat16>(p, back, s)
                    : add_io<float, __nv_bfloat16>(p, back, s);
}

}  // namespace

GDR_DEFINE_OOB_COUNTER(oob_count_norms)

cudaError_t launch_gated_norm_fwd(const GatedNormArgs &p, cudaStream_t s) {
  return p.bf16 ? gated_io<__nv_bfloat16>(p, false, s) : gated_io<float>(p, false, s);
}
cudaError_t launch_gated_norm_bwd(const GatedNormArgs &p, cudaStream_t s) {
  return p.bf16 ? gated_io<__nv_bfloat16>(p, true, s) : gated_io<float>(p, true, s);
}
cudaError_t launch_add_norm_fwd(const AddNormArgs &p, cudaStream_t s) { return add_any(p, false, s); }
cudaError_t launch_add_norm_bwd(const AddNormArgs &p, cudaStream_t s) { return add_any(p, true, s); }

}  // namespace gdr
