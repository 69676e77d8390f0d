// Gated RMS norm, forward and backward (sm_100a).  Per head row x of d channels,
// with weight w and gate z:
//     u = x r,  r = 1 / sqrt(mean(x^2) + eps),   y = u w s(z),  s = z sigmoid(z) | sigmoid(z) | 1
//     du = dy w s,  dx = r (du - u mean(du u)),  dz = dy u w s'(z),  dw = sum over rows of dy u s
// mean(du u) = r mean(du x), so the backward pass takes both of its row sums in
// one reduction.  16384 x 32 x 128 bf16: 68 us (sigmoid) = 5.9 TB/s and 70 (silu);
// gradient 120 = 5.6 TB/s and 133 = 5.0, where the gate's instructions show; fp32 133
// and 224 us = 6.1 and 6.0 TB/s.  Other head sizes are slower: 16384 x 32 x 96 bf16 66
// and 123 us = 4.6 and 4.1 TB/s, 16384 x 16 x 333 175 and 304 = 3.0 and 2.9.
#include "norms.cuh"

namespace gdr {
namespace norms {
namespace {

// sigmoid.  bf16 results keep 8 bits, so the approximations' few ulp are far below
// their rounding (an exponential that overflows gives 0, as it should); fp32 ones
// take the accurate functions.
template <typename IO> __device__ __forceinline__ float2 exp_of_minus(float2 z) {
  if constexpr (sizeof(IO) == 2) {
    const float2 t = mul2(z, both(-1.44269504f));  // -log2 e
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    return e;
  } else {
    return make_float2(expf(-z.x), expf(-z.y));
  }
}
template <typename IO> __device__ __forceinline__ float2 one_over(float2 x) {
  if constexpr (sizeof(IO) == 2) {
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(x.y));
    return r;
  } else {
    return make_float2(1.f / x.x, 1.f / x.y);
  }
}
template <typename IO, bool SILU> __device__ __forceinline__ float2 gate_value(float2 z) {
  const float2 g = one_over<IO>(add2(exp_of_minus<IO>(z), both(1.f)));
  return SILU ? mul2(z, g) : g;
}

// The gate's value and its slope.  1 - g of g = sigmoid(z) is exp(-z) g: as a
// difference it has one digit left at z = 15 in fp32, and none at 17.  (Where the
// exponential overflows, g is 0 and 1 - g of no account.)
__device__ __forceinline__ float finite(float e) {
  asm("min.NaN.f32 %0, %0, 0f7F7FFFFF;" : "+f"(e));
  return e;
}
template <typename IO, bool SILU> __device__ __forceinline__ float2 gate_value(float2 z, float2 &slope) {
  const float2 e = exp_of_minus<IO>(z), g = one_over<IO>(add2(e, both(1.f)));
  const float2 rest = mul2(make_float2(finite(e.x), finite(e.y)), g);
  slope = mul2(g, SILU ? fma2(z, rest, both(1.f)) : rest);
  return SILU ? mul2(z, g) : g;
}

// A row of a [tokens, H, d] tensor whose tokens are ld elements apart, as the group walks.
struct HeadRow {
  int64_t tok, dtok;
  int head, dhead, H;
  __device__ __forceinline__ HeadRow(int64_t row, int64_t step, int H_) : H(H_) {
    tok = (uint32_t)row / (uint32_t)H;  // (rows fit in 31 bits)
    head = (int)(row - tok * H);
    dtok = (uint32_t)step / (uint32_t)H;
    dhead = (int)(step - dtok * H);
  }
  __device__ __forceinline__ void next() {
    tok += dtok;
    head += dhead;
    if (head >= H) {
      head -= H;
      ++tok;
    }
  }
  __device__ __forceinline__ int64_t at(int64_t ld, int d) const { return tok * ld + (int64_t)head * d; }
};

// SILU, or sigmoid and (p.gate) no gate.
template <typename IO, int V, int NV, int LANES, bool ODD, bool SILU>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads<V, false>)
gated_norm_fwd_kernel(const __grid_constant__ GatedNormArgs p) {
  constexpr int NP = Pairs<V>::N;
  __shared__ float2 buf[64];
  extern __shared__ __align__(16) float shared[];
  Group<V, NV, LANES, ODD> grp(buf, p.tokens * p.H, p.d);
  const Columns<V, NV, LANES, ODD, kAgain<V, NV, LANES, ODD>> weight(grp, p.weight, shared);
  const bool gated = SILU || p.gate != KDA_GATE_NONE;
  HeadRow at(grp.row, grp.step, p.H);
  for (int64_t row = grp.row; grp.more(row); row += grp.step, at.next()) {
    const bool live = row < grp.rows;
    Pack<IO, V> x[NV], z[NV];
    float2 ss = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i].zero();
      z[i].zero();
      if (!live || !grp.any[i] || !GDR_IN_BOUNDS(at.tok < p.tokens)) continue;
      x[i].load(static_cast<const IO *>(p.x) + at.at(p.ld_x, p.d), grp.c[i], p.d, grp.inside(i, row));
      if (gated) z[i].load(static_cast<const IO *>(p.z) + at.at(p.ld_z, p.d), grp.c[i], p.d, grp.inside(i, row));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (ODD && !grp.whole[i]) x[i].keep(grp.half[i]);
#pragma unroll
      for (int j = 0; j < NP; ++j) ss = fma2(x[i].pair(j), x[i].pair(j), ss);
    }
    const float2 inv = both(rsqrtf(grp.sum(ss.x + ss.y) / (float)p.d + p.eps));
    IO *y = static_cast<IO *>(p.y) + row * p.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float2 w[NP];
      weight.get(grp, i, w);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        w[j] = mul2(w[j], mul2(x[i].pair(j), inv));
        if (gated) w[j] = mul2(w[j], gate_value<IO, SILU>(z[i].pair(j)));
      }
      if (live && grp.any[i] && GDR_IN_BOUNDS(row < grp.rows)) store_piece<IO, V>(y, grp.c[i], grp.whole[i], grp.half[i], w);
    }
  }
}

// The next row's loads are under way while this one is worked on (few blocks fit
// an SM), as far as a thread has one piece.  Registers for three blocks of warps
// an SM (two with silu in bf16 or with masked pieces, which need more: they would
// spill); for a block a row 80 a thread (65536 over 800), six blocks of 128: 16384
// x 4 x 1000 bf16 118 us, with 82 registers 132.
template <int LANES, int NV, bool ODD> constexpr int kBackThreads =
    LANES ? 256 : NV == 1 && !ODD ? 800 : kMostThreads;
template <typename IO, int V, int NV, int LANES, bool ODD, bool SILU>
__global__ void __launch_bounds__(kBackThreads<LANES, NV, ODD>,
                                  LANES && NV == 1 ? SILU && (sizeof(IO) == 2 || ODD) ? 2 : 3 : 1)
gated_norm_bwd_kernel(const __grid_constant__ GatedNormArgs p) {
  constexpr int NP = Pairs<V>::N;
  let_next_start();
  constexpr bool EARLY = NV == 1;
  __shared__ float2 buf[64];
  extern __shared__ __align__(16) float shared[];
  Group<V, NV, LANES, ODD> grp(buf, p.tokens * p.H, p.d);
  const Columns<V, NV, LANES, ODD, false> weight(grp, p.weight, shared);
  const bool gated = SILU || p.gate != KDA_GATE_NONE;
  HeadRow at(grp.row, grp.step, p.H);
  float2 acc[NV][NP];
  Pack<IO, V> dy[NV], x[NV], z[NV];
  auto load = [&](int64_t row) {
    if (row >= grp.rows) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!grp.any[i] || !GDR_IN_BOUNDS(at.tok < p.tokens)) continue;
      const bool inside = grp.inside(i, row);
      x[i].load(static_cast<const IO *>(p.x) + at.at(p.ld_x, p.d), grp.c[i], p.d, inside);
      dy[i].load(static_cast<const IO *>(p.dy) + at.at(p.ld_dy, p.d), grp.c[i], p.d, inside);
      if (gated) z[i].load(static_cast<const IO *>(p.z) + at.at(p.ld_z, p.d), grp.c[i], p.d, inside);
    }
    at.next();
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i].zero();
    dy[i].zero();
    z[i].zero();
#pragma unroll
    for (int j = 0; j < NP; ++j) acc[i][j] = both(0.f);
  }
  load(grp.row);
  for (int64_t row = grp.row; grp.more(row); row += grp.step) {
    const bool live = row < grp.rows;
    Pack<IO, V> cx[NV];
    float2 t[NV][NP], ds[NV][NP], ss = both(0.f), sd = both(0.f);  // t: dy s; ds: dy s'
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live) {  // (a group past the last row adds nothing, whatever it held; a block never is)
        dy[i].zero();
        if (LANES) z[i].zero();
      }
      cx[i] = x[i];
      Pack<IO, V> cdy = dy[i], cz = z[i];
      if (ODD && !grp.whole[i]) {
        cx[i].keep(grp.half[i]);
        cdy.keep(grp.half[i]);
        cz.keep(grp.half[i]);
      }
      float2 w[NP];
      weight.get(grp, i, w);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const float2 xv = cx[i].pair(j);
        t[i][j] = cdy.pair(j);
        if (gated) {
          float2 slope;
          const float2 g = gate_value<IO, SILU>(cz.pair(j), slope);
          ds[i][j] = mul2(t[i][j], slope);
          t[i][j] = mul2(t[i][j], g);
        }
        ss = fma2(xv, xv, ss);
        sd = fma2(mul2(t[i][j], w[j]), xv, sd);
      }
    }
    if (EARLY) load(row + grp.step);
    const float2 sum = grp.sum(ss.x + ss.y, sd.x + sd.y);
    const float inv = rsqrtf(sum.x / (float)p.d + p.eps);
    const float m = inv * inv * (sum.y / (float)p.d);  // mean(du u) r
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float2 dx[NP], dz[NP], w[NP];
      weight.get(grp, i, w);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const float2 xv = cx[i].pair(j), u = mul2(xv, both(inv));
        dx[j] = mul2(both(inv), fma2(xv, both(-m), mul2(t[i][j], w[j])));
        acc[i][j] = fma2(t[i][j], u, acc[i][j]);
        dz[j] = mul2(mul2(ds[i][j], w[j]), u);
      }
      if (live && grp.any[i] && GDR_IN_BOUNDS(row < grp.rows)) {
        store_piece<IO, V>(static_cast<IO *>(p.dx) + row * p.d, grp.c[i], grp.whole[i], grp.half[i], dx);
        if (gated) store_piece<IO, V>(static_cast<IO *>(p.dz) + row * p.d, grp.c[i], grp.whole[i], grp.half[i], dz);
      }
    }
    if (!EARLY) load(row + grp.step);
  }
  if (p.partial) write_partial(grp, acc, shared, p.partial);
}

template <typename IO, int V, bool ODD, bool SILU, bool BACK>
cudaError_t gated_gate(const GatedNormArgs &p, cudaStream_t s) {
  const Plan q = plan<V, BACK>(p.d, 1, ODD);
  const int64_t rows = p.tokens * p.H;
  int blocks = 0;
  cudaError_t e = cudaErrorInvalidValue;
#define GDR_LAUNCH(NV, LANES)                                                                                   \
  do {                                                                                                          \
    if constexpr (BACK)                                                                                         \
      e = launch_rows<gated_norm_bwd_kernel<IO, V, NV, LANES, ODD, SILU>>("gated_norm_bwd_kernel", p, q, rows, s, &blocks); \
    else                                                                                                        \
      e = launch_rows<gated_norm_fwd_kernel<IO, V, NV, LANES, ODD, SILU>>("gated_norm_fwd_kernel", p, q, rows, s, &blocks); \
  } while (0)
  GDR_NORM_PLAN(q, GDR_LAUNCH);
#undef GDR_LAUNCH
  return BACK && e == cudaSuccess ? sum_columns(p.partial, p.dweight, nullptr, p.d, blocks, s) : e;
}

template <typename IO, int V, bool ODD> cudaError_t gated_vec(const GatedNormArgs &p, bool back, cudaStream_t s) {
  if (p.gate == KDA_GATE_SILU) return back ? gated_gate<IO, V, ODD, true, true>(p, s) : gated_gate<IO, V, ODD, true, false>(p, s);
  return back ? gated_gate<IO, V, ODD, false, true>(p, s) : gated_gate<IO, V, ODD, false, false>(p, s);
}

// 16-byte accesses where every tensor begins on 16 bytes, and either its rows do
// too or its tokens follow each other without a gap.
template <typename IO> cudaError_t gated_io(const GatedNormArgs &p, bool back, cudaStream_t s) {
  constexpr int V = 16 / sizeof(IO);
  const int64_t row = (int64_t)p.H * p.d;
  const bool packed = p.ld_x == row && (!p.z || p.ld_z == row) && (!p.dy || p.ld_dy == row);
  const bool even = p.d % V == 0 && p.ld_x % V == 0 && p.ld_z % V == 0 && p.ld_dy % V == 0;
  const bool wide = (packed || even) && aligned16(p.x) && aligned16(p.z) && aligned16(p.y) && aligned16(p.dy) &&
                    aligned16(p.dx) && aligned16(p.dz);
  if (!wide) return gated_vec<IO, 1, false>(p, back, s);
  return p.d % V == 0 && aligned16(p.weight) ? gated_vec<IO, V, false>(p, back, s) : gated_vec<IO, V, true>(p, back, s);
}

// out[c] = sum of partial[b][c] over the blocks, in a fixed order.  (The partial
// sums are still written when this kernel starts: no __restrict__, no read-only loads.)
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *partial0, float *out0,
                                                          const float *partial1, float *out1, int blocks,
                                                          int d) {
  wait_for_last();
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

}  // namespace

cudaError_t sum_columns(const float *partial, float *out0, float *out1, int d, int blocks, cudaStream_t s) {
  if (!out0 && !out1) return cudaSuccess;
  TraceScope tr("column_sum_kernel", s);
  return launch_behind(column_sum_kernel, dim3((d + 31) / 32, out1 ? 2 : 1), dim3(32, 32), 0, s, partial, out0,
                       partial + (int64_t)kNormBlocks * d, out1, blocks, d);
}

}  // namespace norms

GDR_DEFINE_OOB_COUNTER(oob_count_gated_norm)

cudaError_t launch_gated_norm_fwd(const GatedNormArgs &p, cudaStream_t s) {
  return p.bf16 ? norms::gated_io<__nv_bfloat16>(p, false, s) : norms::gated_io<float>(p, false, s);
}
cudaError_t launch_gated_norm_bwd(const GatedNormArgs &p, cudaStream_t s) {
  return p.bf16 ? norms::gated_io<__nv_bfloat16>(p, true, s) : norms::gated_io<float>(p, true, s);
}

}  // namespace gdr
