// The gated block and its gradients: row kernels and launches.
#pragma once

#include "fused_rows.hpp"
#include "skinny_launch.hpp"

namespace pgemm {

// dst[row][from .. pitch) = 0: the ends of dy's rows meet W rows that read zero,
// and must be finite.
static __global__ void __launch_bounds__(256) zero_tail_kernel(uint16_t *dst, int64_t rows, int from, int pitch) {
  const int n = pitch - from;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * n; i += (int64_t)gridDim.x * 256)
    dst[i / n * pitch + from + i % n] = 0;
}

// dy[m] = [dh up act'(gate) | dh act(gate)] from the projections that the
// forward call kept (GatedEpi), four hidden columns a thread.  Memory bound:
// 14 bytes a hidden value, 10 read and 4 written; 280 us, 5 TB/s, at 8192 x 12288.
// In an epilogue of the forward call it would have to wait for dh, and in a
// product's loads it would be computed once for every tile that reads dy.
template <typename T>
__global__ void __launch_bounds__(256) gated_slope_kernel(const float *__restrict__ saved,
                                                          const uint16_t *__restrict__ dh, uint16_t *__restrict__ dy,
                                                          int64_t M, int F, int64_t py, int act) {
  const int per = (F + 3) / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * per; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per;
    const int c = (int)(i % per) * 4;
    const f32x4 ga = *reinterpret_cast<const f32x4 *>(saved + i * 8);
    const f32x4 up = *reinterpret_cast<const f32x4 *>(saved + i * 8 + 4);
    const uint16_t *s = dh + m * F + c;
    const bool whole = c + 4 <= F;
    if (c == 0) {  // a row's end meets W rows that read zero, and must be finite
      for (int64_t x = 2 * (int64_t)F; x < py; ++x) dy[m * py + x] = 0;
    }
    u32x2 v = {0u, 0u};
    if (whole) {
      v = *reinterpret_cast<const u32x2_any *>(s);
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (c + x < F) v[x / 2] |= (uint32_t)s[x] << (16 * (x % 2));
    }
    f32x4 dg, du;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float d = widen<T>((uint16_t)(v[x / 2] >> (16 * (x % 2))));
      const Activation a = activate_slope(act, ga[x]);
      dg[x] = d * up[x] * a.d;
      du[x] = d * a.a;
    }
    const u32x2 pg = Mfma<T>::pack4(dg[0], dg[1], dg[2], dg[3]);
    const u32x2 pu = Mfma<T>::pack4(du[0], du[1], du[2], du[3]);
    uint16_t *o = dy + m * py + c;
    if (whole) {
      *reinterpret_cast<u32x2_any *>(o) = pg;
      *reinterpret_cast<u32x2_any *>(o + F) = pu;
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (c + x < F) {
          o[x] = (uint16_t)(pg[x / 2] >> (16 * (x % 2)));
          o[F + x] = (uint16_t)(pu[x / 2] >> (16 * (x % 2)));
        }
    }
  }
}

namespace launch_detail {

// x [M][D] and W [2F][D] as the products read them: in place, or padded.
template <typename T>
pgemm_status gated_operands(const GatedCall &c, const GatedPlan &p, const uint16_t **x, const uint16_t **w) {
  *x = c.x;
  *w = c.w;
  if (!p.padded) return PGEMM_OK;
  return pad_operands(x, c.ws + p.x, c.M, w, c.ws + p.w, 2 * c.F, c.D, p.d8, c.stream);
}

inline FusedProduct projections(const GatedCall &c, const GatedPlan &p, const uint16_t *x, const uint16_t *w) {
  FusedProduct g{};
  g.a = FusedOperand{x, nullptr, (int)p.d8, (int)c.M};
  g.b = FusedOperand{w, w + c.F * p.d8, (int)p.d8, (int)c.F};
  g.M = (int)c.M;
  g.N = (int)c.F;
  g.K = (int)p.d8;
  return g;
}

template <typename T>
pgemm_status gated_forward(const GatedCall &c) {
  const GatedPlan p = plan_gated(c.M, c.F, c.D, false, c.saved != nullptr);
  if (p.skinny) {
    SkinnyArgs a{};
    a.x = c.x;
    a.w = c.w;
    a.out = c.h;
    a.M = (int)c.M;
    a.N = (int)c.F;
    a.K = (int)c.D;
    a.act = c.act;
    return launch_skinny<T, true>(a, c.stream, c.dev);
  }
  const uint16_t *x, *w;
  pgemm_status st = gated_operands<T>(c, p, &x, &w);
  if (st != PGEMM_OK) return st;
  return launch_product<T, Lay::KC, Lay::KC, true, GatedEpi>(projections(c, p, x, w), p.forward,
                                                             GatedEpi::Args{c.h, c.saved, c.act}, c.stream, c.dev);
}

template <typename T>
pgemm_status gated_backward(const GatedCall &c) {
  const GatedPlan p = plan_gated(c.M, c.F, c.D, true, false);
  const uint16_t *x, *w;
  pgemm_status st = gated_operands<T>(c, p, &x, &w);
  if (st != PGEMM_OK) return st;
  uint16_t *dy = reinterpret_cast<uint16_t *>(c.ws + p.dy);
  const int64_t F2 = 2 * c.F;
  // dy = [d gate | d up], rounded to T: the products below take 16-bit
  // operands, and one rounding here costs as much as the one of the result
  if (c.M > 0 && F2 > 0) {
    if (c.saved_in) {
      hipLaunchKernelGGL(gated_slope_kernel<T>, dim3(row_grid(c.M * per(c.F, 4))), dim3(256), 0, c.stream, c.saved_in,
                         c.dh, dy, c.M, (int)c.F, p.py, c.act);
      st = launched();
    } else {
      st = launch_product<T, Lay::KC, Lay::KC, true, GatedSlopeEpi>(
          projections(c, p, x, w), p.forward, GatedSlopeEpi::Args{c.dh, dy, p.py, c.act}, c.stream, c.dev);
      if (st == PGEMM_OK && p.py != F2) {
        hipLaunchKernelGGL(zero_tail_kernel, dim3(row_grid(c.M * (p.py - F2))), dim3(256), 0, c.stream, dy, c.M, (int)F2,
                           (int)p.py);
        st = launched();
      }
    }
    if (st != PGEMM_OK) return st;
  }
  // dx = dy W
  FusedProduct g{};
  g.a = FusedOperand{dy, nullptr, (int)p.py, (int)c.M};
  g.b = FusedOperand{w, nullptr, (int)p.d8, (int)c.D};
  g.M = (int)c.M;
  g.N = (int)c.D;
  g.K = (int)F2;
  st = launch_sum<T, Lay::KC, Lay::KR>(g, p.dx, SumEpi::Args{nullptr, 0, 1, 1, {c.dx, c.D, nullptr}}, c.ws + p.part,
                                       c.stream, c.dev);
  if (st != PGEMM_OK) return st;
  // dW = dy^T x
  g.a = FusedOperand{dy, nullptr, (int)p.py, (int)F2};
  g.b = FusedOperand{x, nullptr, (int)p.d8, (int)c.D};
  g.M = (int)F2;
  g.N = (int)c.D;
  g.K = (int)c.M;
  return launch_sum<T, Lay::KR, Lay::KR>(g, p.dw, SumEpi::Args{nullptr, 0, 1, 1, {c.dw, c.D, nullptr}}, c.ws + p.part,
                                         c.stream, c.dev);
}

}  // namespace launch_detail
}  // namespace pgemm
