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

// The maxima behind DyScale, of what is finite (what is not ends where the
// definition has it end).  A wave takes a run of dh, x or W at a time, as they
// lie; the largest sum of squares of a run, times the runs that a row may
// touch, stands for the rows' norms.  A workgroup alone leaves the exponent itself.
// Bound by memory: the 41 MB of 4095 x 1001 x 2731 take 10.4 us.
constexpr int kRangeRun = 4096;   // values
constexpr int kRangeParts = 256;  // workgroups, one a CU
constexpr int kRangeThreads = 1024;
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

static __global__ void __launch_bounds__(kRangeThreads) gated_range_kernel(const uint16_t *__restrict__ dh, int64_t n_dh,
                                                                           const uint16_t *__restrict__ x,
                                                                           const uint16_t *__restrict__ w, float4 *part,
                                                                           DyScale s) {
  constexpr int WAVES = kRangeThreads / 64, U = kRangeRun / 512;
  __shared__ float4 tops[WAVES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n_x = s.rows_x * s.D, n_w = s.rows_w * s.D;
  const int64_t end_d = (n_dh + kRangeRun - 1) / kRangeRun, end_x = end_d + (n_x + kRangeRun - 1) / kRangeRun;
  const int64_t end_w = end_x + (n_w + kRangeRun - 1) / kRangeRun;
  const float touch = (float)((s.D + kRangeRun - 2) / kRangeRun + 1);
  float4 top = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int64_t i = (int64_t)blockIdx.x * WAVES + wave; i < end_w; i += (int64_t)gridDim.x * WAVES) {
    const int kind = i < end_d ? 0 : i < end_x ? 1 : 2;
    const int64_t at = (i - (kind == 0 ? 0 : kind == 1 ? end_d : end_x)) * kRangeRun;
    const uint16_t *from = (kind == 0 ? dh : kind == 1 ? x : w) + at;
    const int64_t n = kind == 0 ? n_dh : kind == 1 ? n_x : n_w;
    const int left = n - at < kRangeRun ? (int)(n - at) : kRangeRun;
    u32x4 v[U];
    if (n >= 8) {  // of the last piece the values before it again: a few counted twice
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = lane * 8 + u * 512;
        v[u] = *reinterpret_cast<const u32x4_any *>(from + (c < left - 8 ? c : left - 8));
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (lane * 8 + u * 512 >= left) v[u] = u32x4{0u, 0u, 0u, 0u};
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = u32x4{0u, 0u, 0u, 0u};
      if (lane < left) v[0][0] = from[lane];
    }
    // twice where the first pass met an infinity or a NaN: without them
    for (int finite = 0; finite < 2; ++finite) {
      if (finite) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            if ((v[u][d] & 0x7C00u) == 0x7C00u) v[u][d] &= 0xFFFF0000u;
            if ((v[u][d] & 0x7C000000u) == 0x7C000000u) v[u][d] &= 0xFFFFu;
          }
      }
      float found;
      if (kind == 0) {
        u16x2 most = {0, 0};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int d = 0; d < 4; ++d) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, v[u][d] & 0x7FFF7FFFu));
        const uint16_t m = most[0] > most[1] ? most[0] : most[1];
        found = m < 0x7C00u ? widen<_Float16>(m) : INFINITY;
      } else {
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const float a = widen<_Float16>((uint16_t)v[u][d]), b = widen<_Float16>((uint16_t)(v[u][d] >> 16));
            sum[d] = __builtin_fmaf(b, b, __builtin_fmaf(a, a, sum[d]));
          }
        found = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) found += __shfl_xor(found, d);
      }
      if (__any(!(found < INFINITY))) continue;
      top = DyScale::top(top, make_float4(kind == 0 ? found : 0.0f, kind == 1 ? found : 0.0f, kind == 2 ? found : 0.0f, 0.0f));
      break;
    }
  }
  top = DyScale::wave_top(top);
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  if (wave != 0) return;
  top = DyScale::wave_top(tops[lane % WAVES]);
  top.y *= touch;
  top.z *= touch;
  if (gridDim.x > 1) {
    if (lane == 0) part[blockIdx.x] = top;
  } else {
    s.seed(DyScale::exponent(top), lane, 64);
  }
}

// dy[m] = [dh up act'(gate) | dh act(gate)] from the projections that the
// forward call kept (GatedEpi), four hidden columns a thread.  Memory bound:
// 14 bytes a hidden value, 10 read and 4 written; 280 us, 5 TB/s, at 8192 x 12288.
// In an epilogue of the forward call it would have to wait for dh, and in a
// product's loads it would be computed once for every tile that reads dy.
template <typename T>
__global__ void __launch_bounds__(256) gated_slope_kernel(const float *__restrict__ saved,
                                                          const uint16_t *__restrict__ dh, uint16_t *__restrict__ dy,
                                                          int64_t M, int F, int64_t py, int act,
                                                          DyScale scale) {
  const int per = (F + 3) / 4;
  const float k = scale.take(threadIdx.x, 256);
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
      const float d = widen<T>((uint16_t)(v[x / 2] >> (16 * (x % 2)))) * k;
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
    return launch_skinny<T>(a, c.stream);
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
  DyScale scale{nullptr, -1, c.dx, c.dw, c.M, F2, c.D};
  const bool seeded = std::is_same_v<T, _Float16> && c.M > 0 && F2 > 0;
  if (c.M > 0 && F2 > 0) {
    if (seeded) {
      // between two rows of tiles' starts in dw, on 16 bytes
      const int64_t at = up_to(c.D * 2, 16), end = (F2 < kSeedStep ? F2 : kSeedStep) * c.D * 2;
      const int64_t runs = per(c.M * c.F, kRangeRun) + per(c.M * c.D, kRangeRun) + per(F2 * c.D, kRangeRun);
      int64_t blocks = per(runs, kRangeThreads / 64);
      if (blocks > kRangeParts) blocks = kRangeParts;
      if (blocks > (end - at) / 16) blocks = (end - at) / 16 > 1 ? (end - at) / 16 : 1;
      float4 *part = reinterpret_cast<float4 *>(reinterpret_cast<char *>(c.dw) + at);
      hipLaunchKernelGGL(gated_range_kernel, dim3((unsigned)blocks), dim3(kRangeThreads), 0, c.stream, c.dh, c.M * c.F, c.x,
                         c.w, part, scale);
      st = launched();
      if (st != PGEMM_OK) return st;
      scale.part = part;
      scale.parts = blocks > 1 ? (int)blocks : 0;
    }
    if (c.saved_in) {
      // each workgroup takes the factor for itself, so not too many (4095 x 2731: 29.4 us
      // in 4096 of them, 31.3 in 2048, 35 in 10926)
      const unsigned grid = row_grid(c.M * per(c.F, 4));
      hipLaunchKernelGGL(gated_slope_kernel<T>, dim3(seeded && grid > 4096 ? 4096 : grid), dim3(256), 0, c.stream, c.saved_in,
                         c.dh, dy, c.M, (int)c.F, p.py, c.act, scale);
      st = launched();
    } else {
      st = launch_product<T, Lay::KC, Lay::KC, true, GatedSlopeEpi>(
          projections(c, p, x, w), p.forward, GatedSlopeEpi::Args{c.dh, dy, p.py, c.act, scale}, c.stream, c.dev);
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
  st = launch_sum<T, Lay::KC, Lay::KR>(g, p.dx, SumEpi::Args{nullptr, 0, 1, 1, {c.dx, c.D, nullptr, seeded}}, c.ws + p.part,
                                       c.stream, c.dev);
  if (st != PGEMM_OK) return st;
  // dW = dy^T x
  g.a = FusedOperand{dy, nullptr, (int)p.py, (int)F2};
  g.b = FusedOperand{x, nullptr, (int)p.d8, (int)c.D};
  g.M = (int)F2;
  g.N = (int)c.D;
  g.K = (int)c.M;
  return launch_sum<T, Lay::KR, Lay::KR>(g, p.dw, SumEpi::Args{nullptr, 0, 1, 1, {c.dw, c.D, nullptr, seeded}}, c.ws + p.part,
                                         c.stream, c.dev);
}

}  // namespace launch_detail
}  // namespace pgemm
