// Residual add and RMS norm, forward and backward (sm_100a):
//     t = residual + scale y,  n = t r w,   u = t r,  r = 1 / sqrt(mean(t^2) + eps)
//     d = dt + r (dn w - u mean(dn w u)),  dresidual = d,  dy = scale d,
//     dw = sum over rows of dn u,  dscale = sum of d y
// 8192 x 4096 with an fp32 residual: 66 us = 6.1 TB/s, gradient 103 = 5.9; in bf16 52
// and 83 us = 5.2 and 4.9 TB/s (a block a row: the sum over it and the
// instructions around it show).  8192 x 4095 bf16: 66 and 99 us.  Gradients of long
// rows spill (more than 10240 channels in bf16, 5120 in fp32): 4096 x 16384 bf16 126 and
// 252 us = 4.3 and 3.2 TB/s, 4096 x 8192 fp32 155 and 510 = 3.5 and 1.6.
#include "norms.cuh"

namespace gdr {
namespace norms {
namespace {

template <typename RES, typename IO, int V, int NV, int LANES, bool ODD>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads<V, false>)
add_norm_fwd_kernel(const __grid_constant__ AddNormArgs p) {
  constexpr int NP = Pairs<V>::N;
  __shared__ float2 buf[64];
  extern __shared__ __align__(16) float shared[];
  Group<V, NV, LANES, ODD> grp(buf, p.rows, p.D);
  const Columns<V, NV, LANES, ODD, kAgain<V, NV, LANES, ODD>> weight(grp, p.weight, column_slots<V, NV, LANES>(shared, 0));
  const Columns<V, NV, LANES, ODD, kAgain<V, NV, LANES, ODD>> scale(grp, p.scale, column_slots<V, NV, LANES>(shared, 1));
  for (int64_t row = grp.row; grp.more(row); row += grp.step) {
    const bool live = row < grp.rows;
    Pack<RES, V> r[NV];
    Pack<IO, V> y[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      r[i].zero();
      y[i].zero();
      if (!live || !grp.any[i] || !GDR_IN_BOUNDS(row < p.rows)) continue;
      r[i].load(static_cast<const RES *>(p.residual) + row * p.D, grp.c[i], p.D, grp.inside(i, row));
      y[i].load(static_cast<const IO *>(p.y) + row * p.D, grp.c[i], p.D, grp.inside(i, row));
    }
    float2 t[NV][NP], ss = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (ODD && !grp.whole[i]) {
        r[i].keep(grp.half[i]);
        y[i].keep(grp.half[i]);
      }
      float2 sc[NP];
      scale.get(grp, i, sc);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        t[i][j] = fma2(sc[j], y[i].pair(j), r[i].pair(j));
        ss = fma2(t[i][j], t[i][j], ss);
      }
      if (live && grp.any[i] && GDR_IN_BOUNDS(row < p.rows))
        store_piece<RES, V>(static_cast<RES *>(p.residual_out) + row * p.D, grp.c[i], grp.whole[i], grp.half[i], t[i]);
    }
    const float2 inv = both(rsqrtf(grp.sum(ss.x + ss.y) / (float)p.D + p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float2 w[NP];
      weight.get(grp, i, w);
#pragma unroll
      for (int j = 0; j < NP; ++j) w[j] = mul2(w[j], mul2(t[i][j], inv));
      if (live && grp.any[i] && GDR_IN_BOUNDS(row < p.rows))
        store_piece<IO, V>(static_cast<IO *>(p.n) + row * p.D, grp.c[i], grp.whole[i], grp.half[i], w);
    }
  }
}

// The next row's loads are under way while this one is worked on (few blocks fit
// an SM), as far as a thread has one piece.
template <typename RES, typename IO, int V, int NV, int LANES, bool ODD>
__global__ void __launch_bounds__(LANES ? 256 : kBlockThreads<V, true>)
add_norm_bwd_kernel(const __grid_constant__ AddNormArgs p) {
  constexpr int NP = Pairs<V>::N;
  let_next_start();
  constexpr bool EARLY = NV == 1;
  __shared__ float2 buf[64];
  extern __shared__ __align__(16) float shared[];
  Group<V, NV, LANES, ODD> grp(buf, p.rows, p.D);
  const bool want_dscale = p.dscale != nullptr;
  const Columns<V, NV, LANES, ODD, false> weight(grp, p.weight, column_slots<V, NV, LANES>(shared, 0));
  const Columns<V, NV, LANES, ODD, false> scale(grp, p.scale, column_slots<V, NV, LANES>(shared, 1));
  float2 aw[NV][NP], as[NV][NP];
  Pack<RES, V> t[NV], dt[NV];
  Pack<IO, V> dn[NV], y[NV];
  auto load = [&](int64_t row) {
    if (row >= grp.rows) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!grp.any[i] || !GDR_IN_BOUNDS(row < p.rows)) continue;
      const bool inside = grp.inside(i, row);
      t[i].load(static_cast<const RES *>(p.residual_out) + row * p.D, grp.c[i], p.D, inside);
      dn[i].load(static_cast<const IO *>(p.dn) + row * p.D, grp.c[i], p.D, inside);
      if (p.dresidual_out)
        dt[i].load(static_cast<const RES *>(p.dresidual_out) + row * p.D, grp.c[i], p.D, inside);
      if (want_dscale) y[i].load(static_cast<const IO *>(p.y) + row * p.D, grp.c[i], p.D, inside);
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    t[i].zero();
    dt[i].zero();
    dn[i].zero();
    y[i].zero();
#pragma unroll
    for (int j = 0; j < NP; ++j) aw[i][j] = as[i][j] = both(0.f);
  }
  load(grp.row);
  for (int64_t row = grp.row; grp.more(row); row += grp.step) {
    const bool live = row < grp.rows;
    Pack<RES, V> ct[NV], cdt[NV];
    Pack<IO, V> cdn[NV], cy[NV];
    float2 ss = both(0.f), sd = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live) {  // (a group past the last row adds nothing, whatever it held; a block never is)
        dn[i].zero();
        y[i].zero();
        if (LANES) dt[i].zero();
      }
      ct[i] = t[i];
      cdt[i] = dt[i];
      cdn[i] = dn[i];
      cy[i] = y[i];
      if (ODD && !grp.whole[i]) {
        ct[i].keep(grp.half[i]);
        cdn[i].keep(grp.half[i]);
      }
      float2 w[NP];
      weight.get(grp, i, w);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const float2 tv = ct[i].pair(j);
        ss = fma2(tv, tv, ss);
        sd = fma2(mul2(cdn[i].pair(j), w[j]), tv, sd);
      }
    }
    if (EARLY) load(row + grp.step);
    const float2 s = grp.sum(ss.x + ss.y, sd.x + sd.y);
    const float inv = rsqrtf(s.x / (float)p.D + p.eps);
    const float m = inv * inv * (s.y / (float)p.D);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float2 d[NP], w[NP];
      weight.get(grp, i, w);
#pragma unroll
      for (int j = 0; j < NP; ++j) {  // (sums of columns that are not the thread's are never written)
        const float2 tv = ct[i].pair(j), gv = cdn[i].pair(j);
        d[j] = fma2(both(inv), fma2(tv, both(-m), mul2(gv, w[j])), cdt[i].pair(j));
        aw[i][j] = fma2(gv, mul2(tv, both(inv)), aw[i][j]);
        as[i][j] = fma2(d[j], cy[i].pair(j), as[i][j]);
      }
      if (live && grp.any[i] && GDR_IN_BOUNDS(row < p.rows)) {
        store_piece<RES, V>(static_cast<RES *>(p.dresidual) + row * p.D, grp.c[i], grp.whole[i], grp.half[i], d);
        if (p.dy) {
          scale.get(grp, i, w);
#pragma unroll
          for (int j = 0; j < NP; ++j) d[j] = mul2(d[j], w[j]);
          store_piece<IO, V>(static_cast<IO *>(p.dy) + row * p.D, grp.c[i], grp.whole[i], grp.half[i], d);
        }
      }
    }
    if (!EARLY) load(row + grp.step);
  }
  if (p.dweight) write_partial(grp, aw, shared, p.partial);
  if (want_dscale) write_partial(grp, as, shared, p.partial + (int64_t)kNormBlocks * p.D);
}

template <typename RES, typename IO, int V, bool ODD, bool BACK>
cudaError_t add_plan(const AddNormArgs &p, cudaStream_t s) {
  const Plan q = plan<V, BACK>(p.D, 2, ODD);
  int blocks = 0;
  cudaError_t e = cudaErrorInvalidValue;
#define GDR_LAUNCH(NV, LANES)                                                                                  \
  do {                                                                                                         \
    if constexpr (BACK)                                                                                        \
      e = launch_rows<add_norm_bwd_kernel<RES, IO, V, NV, LANES, ODD>>("add_norm_bwd_kernel", p, q, p.rows, s, &blocks); \
    else                                                                                                       \
      e = launch_rows<add_norm_fwd_kernel<RES, IO, V, NV, LANES, ODD>>("add_norm_fwd_kernel", p, q, p.rows, s, &blocks); \
  } while (0)
  GDR_NORM_PLAN(q, GDR_LAUNCH);
#undef GDR_LAUNCH
  return BACK && e == cudaSuccess ? sum_columns(p.partial, p.dweight, p.dscale, p.D, blocks, s) : e;
}
template <typename RES, typename IO, int V, bool ODD>
cudaError_t add_vec(const AddNormArgs &p, bool back, cudaStream_t s) {
  return back ? add_plan<RES, IO, V, ODD, true>(p, s) : add_plan<RES, IO, V, ODD, false>(p, s);
}

// 16-byte accesses where every tensor begins on 16 bytes.
template <typename RES, typename IO> cudaError_t add_io(const AddNormArgs &p, bool back, cudaStream_t s) {
  constexpr int V = 16 / sizeof(IO);
  const bool wide = aligned16(p.residual) && aligned16(p.y) && aligned16(p.residual_out) && aligned16(p.n) &&
                    aligned16(p.dn) && aligned16(p.dresidual_out) && aligned16(p.dresidual) && aligned16(p.dy);
  if (!wide) return add_vec<RES, IO, 1, false>(p, back, s);
  return p.D % V == 0 && aligned16(p.weight) && aligned16(p.scale) ? add_vec<RES, IO, V, false>(p, back, s) : add_vec<RES, IO, V, true>(p, back, s);
}

cudaError_t add_any(const AddNormArgs &p, bool back, cudaStream_t s) {
  if (!p.bf16) return add_io<float, float>(p, back, s);
  return p.res_bf16 ? add_io<__nv_bfloat16, __nv_bfloat16>(p, back, s) : add_io<float, __nv_bfloat16>(p, back, s);
}

}  // namespace
}  // namespace norms

GDR_DEFINE_OOB_COUNTER(oob_count_add_norm)

cudaError_t launch_add_norm_fwd(const AddNormArgs &p, cudaStream_t s) { return norms::add_any(p, false, s); }
cudaError_t launch_add_norm_bwd(const AddNormArgs &p, cudaStream_t s) { return norms::add_any(p, true, s); }

}  // namespace gdr
