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
// Every row is read once, held in registers as fp32, and each output written
// once: the kernels are bound by HBM.  mean(du u) = r mean(du x), so the
// backward pass takes both of its row sums in one reduction.  A row belongs to
// a group of threads: 8, 16 or 32 lanes of a warp for short rows, a whole block
// for longer ones.  A thread keeps the same columns for every row it meets, so
// the column sums of the weights' gradients are held in registers, then summed
// over a block's groups and over the blocks in a fixed order (no atomics: the
// same inputs give the same bits).
#include "common.cuh"
#include "internal.h"

namespace gdr {
namespace {

constexpr int kBlockThreads = 512;  // most threads of a block that shares one row

// V adjacent elements as floats, one 16-byte access (two for 8 floats) or one element.
template <typename T, int V> __device__ __forceinline__ void load_vec(const T *p, float *x) {
  if constexpr (V == 1) {
    x[0] = io<T>::load(p);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
    x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4 *>(p + i));
      x[i] = f.x; x[i + 1] = f.y; x[i + 2] = f.z; x[i + 3] = f.w;
    }
  }
}
template <typename T, int V> __device__ __forceinline__ void store_vec(T *p, const float *x) {
  if constexpr (V == 1) {
    io<T>::store(p, x[0]);
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                               pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  }
}

// A group of threads that shares one row: LANES lanes of a warp, or the block (LANES = 0).
template <int LANES> struct Group {
  int lane, index, per_block, size;
  float2 *buf;  // [2][32] shared, block groups only
  int turn;
  __device__ __forceinline__ explicit Group(float2 *shared) : buf(shared), turn(0) {
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
  }
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

// sigmoid.  bf16 results keep 8 bits, so the intrinsics' few ulp are far below
// their rounding; fp32 ones take the accurate functions.
template <typename IO> __device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(IO) == 2) return __fdividef(1.f, 1.f + __expf(-z));
  else return 1.f / (1.f + expf(-z));
}
// the gate's value s and slope ds
template <typename IO, int GATE>
__device__ __forceinline__ void gate_of(float z, float &s, float &ds) {
  if (GATE == KDA_GATE_NONE) {
    s = 1.f;
    ds = 0.f;
  } else {
    const float g = sigmoid<IO>(z);
    s = GATE == KDA_GATE_SILU ? z * g : g;
    ds = GATE == KDA_GATE_SILU ? g * (1.f + z * (1.f - g)) : g * (1.f - g);
  }
}

template <typename IO, int V, int NV, int LANES, int GATE>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads) gated_norm_fwd_kernel(GatedNormArgs p) {
  __shared__ float2 buf[64];
  Group<LANES> grp(buf);
  const int64_t rows = p.tokens * p.H;
  const int64_t step = (int64_t)gridDim.x * grp.per_block;
  float w[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * grp.size + grp.lane) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) w[i][v] = p.weight && c < p.d ? __ldg(p.weight + c + v) : 1.f;
  }
  for (int64_t r0 = (int64_t)blockIdx.x * grp.per_block; r0 < rows; r0 += step) {
    const int64_t r = r0 + grp.index;
    const bool live = r < rows;
    const int64_t tok = live ? r / p.H : 0;
    const int head = live ? (int)(r - tok * p.H) : 0;
    const IO *x = static_cast<const IO *>(p.x) + tok * p.ld_x + (int64_t)head * p.d;
    const IO *z = static_cast<const IO *>(p.z) + tok * p.ld_z + (int64_t)head * p.d;
    IO *y = static_cast<IO *>(p.y) + r * p.d;
    float xv[NV][V], zv[NV][V], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
#pragma unroll
      for (int v = 0; v < V; ++v) xv[i][v] = zv[i][v] = 0.f;
      if (live && c < p.d && GDR_IN_BOUNDS(tok < p.tokens && c + V <= p.d)) {
        load_vec<IO, V>(x + c, xv[i]);
        if (GATE != KDA_GATE_NONE) load_vec<IO, V>(z + c, zv[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) ss = fmaf(xv[i][v], xv[i][v], ss);
    const float inv = rsqrtf(grp.sum(ss, 0.f).x / (float)p.d + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float s, ds;
        gate_of<IO, GATE>(zv[i][v], s, ds);
        out[v] = xv[i][v] * inv * w[i][v] * s;
      }
      if (live && c < p.d && GDR_IN_BOUNDS(r < rows && c + V <= p.d)) store_vec<IO, V>(y + c, out);
    }
  }
}

// Sums acc over the block's groups and writes the block's row of partial sums.
template <int V, int NV, int LANES>
__device__ __forceinline__ void write_partial(const Group<LANES> &grp, const float (&acc)[NV][V],
                                              float *smem, float *partial, int d) {
  if (!partial) return;
  if (LANES == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
      if (c < d && GDR_IN_BOUNDS(c + V <= d && blockIdx.x < kNormBlocks))
        for (int v = 0; v < V; ++v) partial[(int64_t)blockIdx.x * d + c + v] = acc[i][v];
    }
    return;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * grp.size + grp.lane) * V;
    if (c < d)
      for (int v = 0; v < V; ++v) smem[grp.index * d + c + v] = acc[i][v];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float t = 0.f;
    for (int k = 0; k < grp.per_block; ++k) t += smem[k * d + c];
    if (GDR_IN_BOUNDS(blockIdx.x < kNormBlocks)) partial[(int64_t)blockIdx.x * d + c] = t;
  }
}

template <typename IO, int V, int NV, int LANES, int GATE>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads) gated_norm_bwd_kernel(GatedNormArgs p) {
  __shared__ float2 buf[64];
  extern __shared__ float sums[];
  Group<LANES> grp(buf);
  const int64_t rows = p.tokens * p.H;
  const int64_t step = (int64_t)gridDim.x * grp.per_block;
  float w[NV][V], acc[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * grp.size + grp.lane) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[i][v] = p.weight && c < p.d ? __ldg(p.weight + c + v) : 1.f;
      acc[i][v] = 0.f;
    }
  }
  for (int64_t r0 = (int64_t)blockIdx.x * grp.per_block; r0 < rows; r0 += step) {
    const int64_t r = r0 + grp.index;
    const bool live = r < rows;
    const int64_t tok = live ? r / p.H : 0;
    const int64_t off = live ? (r - tok * p.H) * p.d : 0;
    const IO *dy = static_cast<const IO *>(p.dy) + tok * p.ld_dy + off;
    const IO *x = static_cast<const IO *>(p.x) + tok * p.ld_x + off;
    const IO *z = static_cast<const IO *>(p.z) + tok * p.ld_z + off;
    float gv[NV][V], xv[NV][V], zv[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
#pragma unroll
      for (int v = 0; v < V; ++v) gv[i][v] = xv[i][v] = zv[i][v] = 0.f;
      if (live && c < p.d && GDR_IN_BOUNDS(tok < p.tokens && c + V <= p.d)) {
        load_vec<IO, V>(x + c, xv[i]);
        load_vec<IO, V>(dy + c, gv[i]);
        if (GATE != KDA_GATE_NONE) load_vec<IO, V>(z + c, zv[i]);
      }
    }
    float ss = 0.f, sd = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float s, ds;
        gate_of<IO, GATE>(zv[i][v], s, ds);
        ss = fmaf(xv[i][v], xv[i][v], ss);
        sd = fmaf(gv[i][v] * w[i][v] * s, xv[i][v], sd);
      }
    const float2 t = grp.sum(ss, sd);
    const float inv = rsqrtf(t.x / (float)p.d + p.eps);
    const float m = inv * inv * (t.y / (float)p.d);  // mean(du u) r
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
      float dx[V], dz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float s, ds;
        gate_of<IO, GATE>(zv[i][v], s, ds);
        const float u = xv[i][v] * inv, gu = gv[i][v] * u;
        dx[v] = inv * (gv[i][v] * w[i][v] * s - xv[i][v] * m);
        dz[v] = gu * w[i][v] * ds;
        acc[i][v] = fmaf(gu, s, acc[i][v]);
      }
      if (live && c < p.d && GDR_IN_BOUNDS(r < rows && c + V <= p.d)) {
        store_vec<IO, V>(static_cast<IO *>(p.dx) + r * p.d + c, dx);
        if (GATE != KDA_GATE_NONE) store_vec<IO, V>(static_cast<IO *>(p.dz) + r * p.d + c, dz);
      }
    }
  }
  write_partial<V, NV, LANES>(grp, acc, sums, p.partial, p.d);
}

template <typename RES, typename IO, int V, int NV, int LANES>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads) add_norm_fwd_kernel(AddNormArgs p) {
  __shared__ float2 buf[64];
  Group<LANES> grp(buf);
  const int64_t step = (int64_t)gridDim.x * grp.per_block;
  for (int64_t r0 = (int64_t)blockIdx.x * grp.per_block; r0 < p.rows; r0 += step) {
    const int64_t r = r0 + grp.index;
    const bool live = r < p.rows;
    float tv[NV][V], yv[NV][V], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
#pragma unroll
      for (int v = 0; v < V; ++v) tv[i][v] = yv[i][v] = 0.f;
      if (live && c < p.D && GDR_IN_BOUNDS(r < p.rows && c + V <= p.D)) {
        load_vec<RES, V>(static_cast<const RES *>(p.residual) + r * p.D + c, tv[i]);
        load_vec<IO, V>(static_cast<const IO *>(p.y) + r * p.D + c, yv[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
      const bool in = live && c < p.D;
      float sc[V];
#pragma unroll
      for (int v = 0; v < V; ++v) sc[v] = 1.f;
      if (in && p.scale) load_vec<float, V>(p.scale + c, sc);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        tv[i][v] = fmaf(sc[v], yv[i][v], tv[i][v]);
        ss = fmaf(tv[i][v], tv[i][v], ss);
      }
      if (in && GDR_IN_BOUNDS(c + V <= p.D))
        store_vec<RES, V>(static_cast<RES *>(p.residual_out) + r * p.D + c, tv[i]);
    }
    const float inv = rsqrtf(grp.sum(ss, 0.f).x / (float)p.D + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
      if (live && c < p.D && GDR_IN_BOUNDS(c + V <= p.D)) {
        float w[V], out[V];
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] = 1.f;
        if (p.weight) load_vec<float, V>(p.weight + c, w);
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = tv[i][v] * inv * w[v];
        store_vec<IO, V>(static_cast<IO *>(p.n) + r * p.D + c, out);
      }
    }
  }
}

template <typename RES, typename IO, int V, int NV, int LANES>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads) add_norm_bwd_kernel(AddNormArgs p) {
  __shared__ float2 buf[64];
  extern __shared__ float sums[];
  Group<LANES> grp(buf);
  const int64_t step = (int64_t)gridDim.x * grp.per_block;
  const bool want_dscale = p.dscale != nullptr;
  float aw[NV][V], as[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) aw[i][v] = as[i][v] = 0.f;
  for (int64_t r0 = (int64_t)blockIdx.x * grp.per_block; r0 < p.rows; r0 += step) {
    const int64_t r = r0 + grp.index;
    const bool live = r < p.rows;
    float tv[NV][V], gv[NV][V], dv[NV][V], yv[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
#pragma unroll
      for (int v = 0; v < V; ++v) tv[i][v] = gv[i][v] = dv[i][v] = yv[i][v] = 0.f;
      if (live && c < p.D && GDR_IN_BOUNDS(r < p.rows && c + V <= p.D)) {
        load_vec<RES, V>(static_cast<const RES *>(p.residual_out) + r * p.D + c, tv[i]);
        load_vec<IO, V>(static_cast<const IO *>(p.dn) + r * p.D + c, gv[i]);
        if (p.dresidual_out)
          load_vec<RES, V>(static_cast<const RES *>(p.dresidual_out) + r * p.D + c, dv[i]);
        if (want_dscale) load_vec<IO, V>(static_cast<const IO *>(p.y) + r * p.D + c, yv[i]);
      }
    }
    float ss = 0.f, sd = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
      float w[V];
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] = 1.f;
      if (p.weight && c < p.D) load_vec<float, V>(p.weight + c, w);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        ss = fmaf(tv[i][v], tv[i][v], ss);
        sd = fmaf(gv[i][v] * w[v], tv[i][v], sd);
      }
    }
    const float2 t = grp.sum(ss, sd);
    const float inv = rsqrtf(t.x / (float)p.D + p.eps);
    const float m = inv * inv * (t.y / (float)p.D);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * grp.size + grp.lane) * V;
      if (live && c < p.D && GDR_IN_BOUNDS(c + V <= p.D)) {
        float w[V], d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] = 1.f;
        if (p.weight) load_vec<float, V>(p.weight + c, w);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          d[v] = dv[i][v] + inv * (gv[i][v] * w[v] - tv[i][v] * m);
          aw[i][v] = fmaf(gv[i][v], tv[i][v] * inv, aw[i][v]);
          as[i][v] = fmaf(d[v], yv[i][v], as[i][v]);
        }
        store_vec<RES, V>(static_cast<RES *>(p.dresidual) + r * p.D + c, d);
        if (p.dy) {
          float sc[V];
#pragma unroll
          for (int v = 0; v < V; ++v) sc[v] = 1.f;
          if (p.scale) load_vec<float, V>(p.scale + c, sc);
#pragma unroll
          for (int v = 0; v < V; ++v) d[v] *= sc[v];
          store_vec<IO, V>(static_cast<IO *>(p.dy) + r * p.D + c, d);
        }
      }
    }
  }
  if (p.dweight) write_partial<V, NV, LANES>(grp, aw, sums, p.partial, p.D);
  if (want_dscale)
    write_partial<V, NV, LANES>(grp, as, sums, p.partial + (int64_t)kNormBlocks * p.D, p.D);
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
  int lanes, nv, threads, blocks;  // lanes 0: a block a row
  size_t smem;                     // for the column sums
};
// Rows of up to 32 vectors go to the 8, 16 or 32 lanes of a warp that hold one
// vector each, longer ones to a block with one vector a thread, up to 512
// threads, and more vectors a thread only beyond that.
Plan plan(int64_t rows, int d, int V) {
  Plan q{};
  const int vecs = (d + V - 1) / V;
  if (vecs <= 32) {
    q.lanes = vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32;
    q.nv = 1;
    q.threads = 256;
    q.smem = (size_t)(q.threads / q.lanes) * d * sizeof(float);
  } else {
    q.lanes = 0;
    q.nv = 1;
    while ((vecs + q.nv - 1) / q.nv > kBlockThreads) q.nv *= 2;
    q.threads = ((vecs + q.nv - 1) / q.nv + 31) / 32 * 32;
  }
  const int per = q.lanes ? q.threads / q.lanes : 1;
  const int64_t want = (rows + per - 1) / per;
  q.blocks = (int)(want < kNormBlocks ? want : kNormBlocks);
  return q;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define GDR_NORM_LANES(q, LAUNCH)                                   \
  do {                                                              \
    if (q.lanes == 8) LAUNCH(1, 8);                                 \
    else if (q.lanes == 16) LAUNCH(1, 16);                          \
    else if (q.lanes == 32) LAUNCH(1, 32);                          \
    else if (q.nv == 1) LAUNCH(1, 0);                               \
    else if (q.nv == 2) LAUNCH(2, 0);                               \
    else if (q.nv == 4) LAUNCH(4, 0);                               \
    else if (q.nv == 8) LAUNCH(8, 0);                               \
    else if constexpr (V == 1) {                                    \
      if (q.nv == 16) LAUNCH(16, 0);                                \
      else LAUNCH(32, 0);                                           \
    }                                                               \
  } while (0)
static_assert(kNormMaxRow <= kBlockThreads * 32, "a block of 512 threads holds the longest row");

template <typename IO, int V, int GATE>
cudaError_t gated_gate(const GatedNormArgs &p, bool back, cudaStream_t s) {
  const Plan q = plan(p.tokens * p.H, p.d, V);
  if (!back) {
    TraceScope tr("gated_norm_fwd_kernel", s);
#define GDR_LAUNCH(NV, LANES) gated_norm_fwd_kernel<IO, V, NV, LANES, GATE><<<q.blocks, q.threads, 0, s>>>(p)
    GDR_NORM_LANES(q, GDR_LAUNCH);
#undef GDR_LAUNCH
    return cudaGetLastError();
  }
  {
    TraceScope tr("gated_norm_bwd_kernel", s);
#define GDR_LAUNCH(NV, LANES) gated_norm_bwd_kernel<IO, V, NV, LANES, GATE><<<q.blocks, q.threads, q.smem, s>>>(p)
    GDR_NORM_LANES(q, GDR_LAUNCH);
#undef GDR_LAUNCH
  }
  if (p.dweight) {
    TraceScope tr("column_sum_kernel", s);
    column_sum_kernel<<<dim3((p.d + 31) / 32, 1), dim3(32, 32), 0, s>>>(p.partial, p.dweight, nullptr,
                                                                       nullptr, q.blocks, p.d);
  }
  return cudaGetLastError();
}

template <typename IO, int V> cudaError_t gated_vec(const GatedNormArgs &p, bool back, cudaStream_t s) {
  switch (p.gate) {
    case KDA_GATE_SILU: return gated_gate<IO, V, KDA_GATE_SILU>(p, back, s);
    case KDA_GATE_SIGMOID: return gated_gate<IO, V, KDA_GATE_SIGMOID>(p, back, s);
    default: return gated_gate<IO, V, KDA_GATE_NONE>(p, back, s);
  }
}

// 16-byte accesses where every row of every tensor begins on 16 bytes.
template <typename IO> cudaError_t gated_io(const GatedNormArgs &p, bool back, cudaStream_t s) {
  constexpr int V = 16 / sizeof(IO);
  const bool wide = p.d % V == 0 && p.ld_x % V == 0 && p.ld_z % V == 0 && p.ld_dy % V == 0 &&
                    aligned16(p.x) && aligned16(p.z) && aligned16(p.y) && aligned16(p.dy) &&
                    aligned16(p.dx) && aligned16(p.dz);
  return wide ? gated_vec<IO, V>(p, back, s) : gated_vec<IO, 1>(p, back, s);
}

template <typename RES, typename IO, int V>
cudaError_t add_vec(const AddNormArgs &p, bool back, cudaStream_t s) {
  const Plan q = plan(p.rows, p.D, V);
  if (!back) {
    TraceScope tr("add_norm_fwd_kernel", s);
#define GDR_LAUNCH(NV, LANES) add_norm_fwd_kernel<RES, IO, V, NV, LANES><<<q.blocks, q.threads, 0, s>>>(p)
    GDR_NORM_LANES(q, GDR_LAUNCH);
#undef GDR_LAUNCH
    return cudaGetLastError();
  }
  {
    TraceScope tr("add_norm_bwd_kernel", s);
#define GDR_LAUNCH(NV, LANES) add_norm_bwd_kernel<RES, IO, V, NV, LANES><<<q.blocks, q.threads, q.smem, s>>>(p)
    GDR_NORM_LANES(q, GDR_LAUNCH);
#undef GDR_LAUNCH
  }
  if (p.dweight || p.dscale) {
    TraceScope tr("column_sum_kernel", s);
    column_sum_kernel<<<dim3((p.D + 31) / 32, 2), dim3(32, 32), 0, s>>>(
        p.partial, p.dweight, p.partial + (int64_t)kNormBlocks * p.D, p.dscale, q.blocks, p.D);
  }
  return cudaGetLastError();
}

template <typename RES, typename IO> cudaError_t add_io(const AddNormArgs &p, bool back, cudaStream_t s) {
  constexpr int V = 16 / sizeof(IO);
  const bool wide = p.D % V == 0 && aligned16(p.residual) && aligned16(p.y) && aligned16(p.scale) &&
                    aligned16(p.weight) && aligned16(p.residual_out) && aligned16(p.n) &&
                    aligned16(p.dn) && aligned16(p.dresidual_out) && aligned16(p.dresidual) &&
                    aligned16(p.dy);
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
