// What the norm kernels share (sm_100a): rows in 16-byte pieces, groups of threads
// that hold a row each, the vectors over a row's columns, and column sums.
//
// Every row is read once, held in registers and each output written once: the
// kernels are bound by HBM, and next to it by their instructions, so arithmetic is
// on pairs of elements (packed fp32).  A row belongs to a group of threads: 8, 16
// or 32 lanes of a warp for short rows, a whole block for longer ones.
//
// Accesses are 16 bytes wide on 16-byte boundaries of the whole tensor, whatever
// the row length: a row that begins `shift` elements past a boundary is cut there
// (its first and last pieces are then partial: read whole and cleared at use,
// written element by element).  A group's rows are whole periods of the shifts (8
// rows at most) apart, so its shift, and with it the columns of each thread, stay the same: the column
// sums of the weights' gradients are held in registers, then summed over a block's
// groups and over the blocks in a fixed order (no atomics: the same inputs give
// the same bits).
#pragma once

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace gdr {
namespace norms {

// Most threads of a block that shares one row.  Forward few, with more pieces each:
// more rows fit an SM (a thread's addresses and counters cost as many registers as
// a piece).  Backward, with column sums in registers too, one piece each and the
// next row's loads under way was faster (8192 x 4096 bf16: 82 us, with two pieces
// 111, with two rows under way 89; the loads through shared memory instead of
// registers: 76, but 146 against 107 with an fp32 residual).
template <int V, bool BACK> constexpr int kBlockThreads = V == 1 || BACK ? 640 : 288;
constexpr int kMostThreads = 640;
constexpr int kCachedDevices = 64;

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

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
  __device__ __forceinline__ float2 pair(int j) const {
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(word(2 * j)), __uint_as_float(word(2 * j + 1)));
    else return make_float2(bf16_lo(word(j)), bf16_hi(word(j)));
  }
  // `inside`: the piece lies in the tensor; else its elements with 0 <= c + v < d
  // do.  What it holds of other rows is cleared by keep().  (Plain loads: some
  // callers write the tensor that they read, row by row.)
  __device__ __forceinline__ void load(const T *row, int c, int d, bool inside) {
    const T *p = row + c;
    if (inside) {
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
  // clears what `half`, a 16-bit mask an element, does not keep
  __device__ __forceinline__ void keep(const uint32_t (&half)[V / 2]) {
    uint32_t w[4 * N];
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) {
      if constexpr (sizeof(T) == 2) w[i] = word(i) & half[i];
      else w[i] = word(i) & (uint32_t)(i & 1 ? (int)half[i / 2] >> 16 : (int)(half[i / 2] << 16) >> 16);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
};
template <typename T> struct Pack<T, 1> {
  T r;
  __device__ __forceinline__ void zero() { r = T(0.f); }
  __device__ __forceinline__ float2 pair(int) const { return make_float2(float(r), 0.f); }
  __device__ __forceinline__ void load(const T *row, int c, int, bool) { r = row[c]; }
  __device__ __forceinline__ void keep(const uint32_t (&)[1]) {}
};
// pairs of a piece
template <int V> struct Pairs {
  static constexpr int N = (V + 1) / 2;
};

// Stores a piece: all of it, or the elements that `half` keeps.
template <typename T, int V>
__device__ __forceinline__ void store_piece(T *row, int c, bool whole, const uint32_t (&half)[(V + 1) / 2],
                                            const float2 (&x)[Pairs<V>::N]) {
  T *p = row + c;
  if constexpr (V == 1) {
    io<T>::store(p, x[0].x);
  } else {
    constexpr int W = V * sizeof(T) / 4;
    uint32_t w[W];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      if constexpr (sizeof(T) == 4) {
        w[2 * j] = __float_as_uint(x[j].x);
        w[2 * j + 1] = __float_as_uint(x[j].y);
      } else {
        w[j] = pack_bf16x2(x[j].x, x[j].y);
      }
    }
    if (whole) {
#pragma unroll
      for (int i = 0; i < W / 4; ++i)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (half[v / 2] >> 16 * (v & 1) & 1) {
          if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t *>(p)[v] = w[v];
          else reinterpret_cast<unsigned short *>(p)[v] = (unsigned short)(w[v / 2] >> 16 * (v & 1));
        }
    }
  }
}

// A group of threads that shares one row: LANES lanes of a warp, or the block
// (LANES = 0); and its walk over the rows.  ODD: rows may begin and end inside a
// piece.
template <int V, int NV, int LANES, bool ODD> struct Group {
  int lane, index, per_block, size, d;
  int64_t row, step, rows;
  int c[NV];  // first column of each of the thread's pieces, and what they are
  bool any[NV], whole[NV];
  uint32_t half[NV][(V + 1) / 2];  // ODD: a 16-bit mask of the row's own elements
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
    const int shift = ODD ? (int)((row % V) * (d % V) % V) : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      c[i] = (i * size + lane) * V - shift;
      any[i] = c[i] < d;
      whole[i] = !ODD || (c[i] >= 0 && c[i] + V <= d);
#pragma unroll
      for (int j = 0; j < (V + 1) / 2; ++j)
        half[i][j] = (in(i, 2 * j) ? 0x0000ffffu : 0u) | (in(i, 2 * j + 1) ? 0xffff0000u : 0u);
    }
  }
  // rows that the block walks: every group takes part in every step's sums
  __device__ __forceinline__ bool more(int64_t r) const { return r - index < rows; }
  // whether a piece of row r lies in a tensor whose rows follow each other (a
  // partial one may run past its end; none runs past its beginning)
  __device__ __forceinline__ bool inside(int i, int64_t r) const {
    return !ODD || whole[i] || r * d + c[i] + V <= rows * d;
  }
  __device__ __forceinline__ bool in(int i, int v) const {
    return ODD ? c[i] + v >= 0 && c[i] + v < d : any[i];
  }
  // Sums over the group, the same bits in each of its threads.  Every thread of
  // the block calls them as often as every other.
  static __device__ __forceinline__ float join(float v, int from) {
#pragma unroll
    for (int o = from; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ __forceinline__ float sum(float a) {
    a = join(a, (LANES ? LANES : 32) / 2);
    return LANES ? a : over_warps(make_float2(a, 0.f), false).x;
  }
  __device__ __forceinline__ float2 sum(float a, float b) {
    if constexpr (LANES != 0) {  // each half of the lanes sums one, then they exchange
      constexpr int kHalf = LANES / 2;
      const bool up = threadIdx.x & kHalf;
      float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, kHalf);
      v = join(v, kHalf / 2);
      const float other = __shfl_xor_sync(0xffffffffu, v, kHalf);
      return up ? make_float2(other, v) : make_float2(v, other);
    }
    // (for a block, whose barrier waits for the slowest warp, two sums side by side
    // were faster: 5001 x 4095 bf16 backward 67.6 us, by halves 69.7)
    return over_warps(make_float2(join(a, 16), join(b, 16)), true);
  }
  // of the warps' sums
  __device__ __forceinline__ float2 over_warps(float2 t, bool two) {
    const int l = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float2 *s = buf + 32 * turn;
    turn ^= 1;
    if (l == 0) s[w] = t;
    __syncthreads();
    t = l < warps ? s[l] : make_float2(0.f, 0.f);
    return make_float2(join(t.x, 16), two ? join(t.y, 16) : 0.f);
  }
};

// A thread's columns of a [d] vector (ones where there is none), the same for
// every row: in registers for the lanes of a warp; for a block in a shared-memory
// slot of the thread's own (no barrier: nobody else reads it), or AGAIN from global
// memory for each row (they stay in L1; 66 against 73 us forward, 8192 x 4096 with
// two pieces a thread, slower with more and backward).
template <int V, int NV, int LANES, bool ODD, bool AGAIN> struct Columns {
  static constexpr int NP = Pairs<V>::N;
  float2 r[LANES ? NV : 1][NP];
  float *slot;
  const float *from;
  __device__ __forceinline__ Columns(const Group<V, NV, LANES, ODD> &grp, const float *p, float *shared) {
    from = p;
    slot = shared + threadIdx.x * V;
    if (AGAIN) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float x = p && grp.in(i, v) ? __ldg(p + grp.c[i] + v) : 1.f;
        if (!LANES) slot[i * (int)blockDim.x * V + v] = x;
        else if (v & 1) r[LANES ? i : 0][v / 2].y = x;
        else r[LANES ? i : 0][v / 2].x = x;
      }
  }
  __device__ __forceinline__ void get(const Group<V, NV, LANES, ODD> &grp, int i, float2 (&x)[NP]) const {
    if (LANES) {
#pragma unroll
      for (int j = 0; j < NP; ++j) x[j] = r[LANES ? i : 0][j];
    } else if constexpr (V == 1) {
      x[0] = make_float2(slot[i * (int)blockDim.x], 0.f);
    } else {
#pragma unroll
      for (int j = 0; j < NP; j += 2) {
        float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
        if (!AGAIN) f = *reinterpret_cast<const float4 *>(slot + i * (int)blockDim.x * V + 2 * j);
        else if (from && grp.any[i]) f = __ldg(reinterpret_cast<const float4 *>(from + grp.c[i] + 2 * j));
        x[j] = make_float2(f.x, f.y);
        x[j + 1] = make_float2(f.z, f.w);
      }
    }
  }
};
template <int V, int NV, int LANES, bool ODD> constexpr bool kAgain = !LANES && !ODD && V > 1 && NV == 2;
// shared memory of the k-th such vector of a block
template <int V, int NV, int LANES> __device__ __forceinline__ float *column_slots(float *shared, int k) {
  return LANES ? shared : shared + (size_t)k * NV * blockDim.x * V;
}

// Sums acc over the block's groups and writes the block's row of partial sums.
template <int V, int NV, int LANES, bool ODD>
__device__ __forceinline__ void write_partial(const Group<V, NV, LANES, ODD> &grp,
                                              const float2 (&acc)[NV][Pairs<V>::N], float *smem, float *partial) {
  const int d = grp.d;
  float *to = LANES ? smem + grp.index * ((d + 3) / 4 * 4) : partial + (int64_t)blockIdx.x * d;
  if (LANES) __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (grp.in(i, v) && GDR_IN_BOUNDS(blockIdx.x < kNormBlocks))
        to[grp.c[i] + v] = v & 1 ? acc[i][v / 2].y : acc[i][v / 2].x;
  if (!LANES) return;
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float t = 0.f;
    for (int k = 0; k < grp.per_block; ++k) t += smem[k * ((d + 3) / 4 * 4) + c];
    if (GDR_IN_BOUNDS(blockIdx.x < kNormBlocks)) partial[(int64_t)blockIdx.x * d + c] = t;
  }
}

struct Plan {
  int lanes, nv, threads;  // lanes 0: a block a row
  int period;              // rows after which their shifts repeat
  size_t smem;             // the columns of the kernel's vectors (a block), or the groups' column sums
};
// Pieces a thread of a block (the last: as many as the longest row needs).
template <int V, bool BACK> struct Pieces {
  static constexpr int a = V == 1 || BACK ? 1 : 2, b = V == 1 ? 4 : BACK ? 2 : 4,
                       c = V == 1 ? 32 : V == 8 ? BACK ? 4 : 8 : BACK ? 8 : 16;
  static_assert(kNormMaxRow + V <= kBlockThreads<V, BACK> * V * c || V == 1, "a block holds the longest row");
};
static_assert(kNormMaxRow <= kBlockThreads<1, false> * 32, "a block holds the longest row");
// Rows of up to 32 pieces go to the 8, 16 or 32 lanes of a warp that hold one
// piece each, of up to 64 forward to a warp with two, longer ones to a block
// (backward a block of two warps with one piece and the next row's loads under way
// is faster: 65536 x 512 bf16 78 us, a warp with two 88).  `vectors`: that the
// kernel keeps the columns of.
template <int V, bool BACK> Plan plan(int d, int vectors, bool odd) {
  Plan q{};
  const int vecs = d % V == 0 ? d / V : (d + 2 * V - 2) / V;  // pieces of a row that begins anywhere
  q.nv = 1;
  for (q.period = 1; q.period * (d % V) % V != 0;) q.period *= 2;
  if (vecs <= (BACK ? 32 : 64)) {
    q.lanes = V == 1 ? 32 : vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32;
    q.nv = vecs <= 32 ? 1 : 2;
    q.threads = 256;
    q.smem = BACK ? (size_t)(q.threads / q.lanes) * ((d + 3) / 4 * 4) * sizeof(float) : 0;
  } else {
    using P = Pieces<V, BACK>;
    const int more[3] = {P::a, P::b, P::c};
    for (int k = 0; k < 3; ++k) {
      q.nv = more[k];
      if ((vecs + q.nv - 1) / q.nv <= kBlockThreads<V, BACK>) break;
    }
    q.threads = ((vecs + q.nv - 1) / q.nv + 31) / 32 * 32;
    q.smem = !BACK && !odd && V > 1 && q.nv == 2 ? 0 : (size_t)vectors * q.nv * q.threads * V * sizeof(float);
  }
  return q;
}
// (227 KB, less the kernels' static part)
constexpr int kMostShared = 227 * 1024 - 1024;

// LAUNCH(pieces a thread, lanes) of a plan
#define GDR_NORM_PLAN(q, LAUNCH)                          \
  do {                                                    \
    using P = Pieces<V, BACK>;                            \
    if (q.lanes == 32 && (BACK || q.nv == 1)) LAUNCH(1, 32); \
    else if (q.lanes == 32) LAUNCH(BACK ? 1 : 2, 32);     \
    else if (q.lanes == 0) {                              \
      if (q.nv == P::a) LAUNCH(P::a, 0);                  \
      else if (q.nv == P::b) LAUNCH(P::b, 0);             \
      else LAUNCH(P::c, 0);                               \
    } else if constexpr (V > 1) {                         \
      if (q.lanes == 8) LAUNCH(1, 8);                     \
      else LAUNCH(1, 16);                                 \
    }                                                     \
  } while (0)

// Blocks that run at once on the current device for this kernel and plan (asked
// once a device and block size).
template <auto KERNEL> cudaError_t resident_blocks(const Plan &q, int *blocks) {
  static std::atomic<int> cache[kCachedDevices][kMostThreads / 32 + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int> *slot = dev >= 0 && dev < kCachedDevices ? &cache[dev][q.threads / 32] : nullptr;
  *blocks = slot ? slot->load(std::memory_order_relaxed) : 0;
  if (*blocks > 0) return cudaSuccess;
  int per_sm = 0;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERNEL, q.threads, q.smem);
  if (e != cudaSuccess) return e;
  *blocks = sm_count() * (per_sm > 0 ? per_sm : 1);
  if (slot) slot->store(*blocks, std::memory_order_relaxed);
  return cudaSuccess;
}

// Launches a norm kernel over `rows` rows; `blocks` becomes its grid.  A group's
// rows are `blocks` times its block's groups apart: a multiple of the period of
// the rows' shifts where a group has more than one (all 148 blocks of a full
// grid where that is 4 or less, else 144).
template <auto KERNEL, typename ARGS>
cudaError_t launch_rows(const char *name, const ARGS &p, const Plan &q, int64_t rows, cudaStream_t s, int *blocks) {
  int most = 0;
  cudaError_t e = resident_blocks<KERNEL>(q, &most);
  if (e != cudaSuccess) return e;
  if (most > kNormBlocks) most = kNormBlocks;
  if (most >= q.period) most -= most % q.period;
  const int per = q.lanes ? q.threads / q.lanes : 1;
  const int64_t want = (rows + per - 1) / per;
  *blocks = (int)(want < most ? want : most);
  TraceScope tr(name, s);
  KERNEL<<<*blocks, q.threads, q.smem, s>>>(p);
  return cudaGetLastError();
}
static_assert(kNormBlocks % 8 == 0, "a full grid keeps the groups' shifts");

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// out0 (out1) = the columns' sums of the first (second) `blocks` rows of partial
// sums, kNormBlocks rows apart.
cudaError_t sum_columns(const float *partial, float *out0, float *out1, int d, int blocks, cudaStream_t s);

}  // namespace norms
}  // namespace gdr
