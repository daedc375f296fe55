// The cross entropy and its gradients: row kernels and launches.
#pragma once

#include "fused_rows.hpp"

namespace pgemm {

// Joins the tiles' softmax statistics of 16 rows per workgroup: 64 threads a
// row run through every 64th part, then theirs are joined.
//   lse = log sum_v e^(z_v), loss = lse - z_target (0 for an ignored row, NaN
// for a target outside the vocabulary).  Bound by memory: 512 parts of 8192 rows
// take 8.8 us, 3.8 TB/s.
template <typename T>
__global__ void __launch_bounds__(1024) lse_join_kernel(const float2 *__restrict__ part, const float *__restrict__ at,
                                                        const int64_t *__restrict__ target, float *__restrict__ loss,
                                                        float *__restrict__ lse, int64_t M, int64_t V, int parts,
                                                        int64_t ignore) {
  __shared__ float tops[16][16], sums[16][16];
  const int r = threadIdx.x & 15, w = threadIdx.x >> 6;
  float top, sum;
  auto join = [&](float t, float s) {
    const float m = fmaxf(top, t);
    const float ref = m == -INFINITY ? 0.0f : m;
    sum = sum * fast_exp(top - ref) + s * fast_exp(t - ref);
    top = m;
  };
  for (int64_t row0 = (int64_t)blockIdx.x * 16; row0 < M; row0 += (int64_t)gridDim.x * 16) {
    const int64_t row = row0 + r;
    top = -INFINITY;
    sum = 0.0f;
    if (row < M) {
#pragma unroll 4
      for (int p = threadIdx.x >> 4; p < parts; p += 64) {
        const float2 v = part[(int64_t)p * M + row];
        join(v.x, v.y);
      }
    }
#pragma unroll
    for (int d = 16; d <= 32; d *= 2) {
      const float t = __shfl_xor(top, d), s = __shfl_xor(sum, d);
      join(t, s);
    }
    if ((threadIdx.x & 63) < 16) {
      tops[w][r] = top;
      sums[w][r] = sum;
    }
    __syncthreads();
    if (threadIdx.x < 16 && row < M) {
#pragma unroll
      for (int p = 1; p < 16; ++p) join(tops[p][r], sums[p][r]);
      const float l = top + logf(sum);
      const int64_t t = target[row];
      lse[row] = l;
      loss[row] = t == ignore ? 0.0f : (t < 0 || t >= V) ? NAN : l - at[row];
    }
    __syncthreads();  // the next rows' go to the same place
  }
}

// scale[0] = the largest finite |dloss| of the rows that count (1 if there is
// none: an infinite one is its own row's matter), scale[1] = scale[0] / kDzUnit<T>: see SlopeEpi.  One
// workgroup, bound by its launch and one trip to memory: 4.6 us for 8192 rows.
template <typename T>
__global__ void __launch_bounds__(1024) loss_scale_kernel(const float *__restrict__ dloss, int dstep,
                                                          const int64_t *__restrict__ target, int64_t M, int64_t ignore,
                                                          float *__restrict__ scale) {
  __shared__ float tops[16];
  float top = 0.0f;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < M; i += 1024) {
    const float d = fabsf(dloss[i * dstep]);
    top = fmaxf(top, target[i] != ignore && d < INFINITY ? d : 0.0f);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 16; ++i) top = fmaxf(top, tops[i]);
    if (top == 0.0f) top = 1.0f;
    scale[0] = top;
    scale[1] = top / kDzUnit<T>;
  }
}

namespace launch_detail {

template <typename T>
pgemm_status xent_operands(const XentCall &c, const XentPlan &p, const uint16_t **x, const uint16_t **w) {
  *x = c.x;
  *w = c.w;
  if (!p.padded) return PGEMM_OK;
  return pad_operands(x, c.ws + p.x, c.M, w, c.ws + p.w, c.V, c.D, p.d8, c.stream);
}

template <typename T>
pgemm_status xent_forward(const XentCall &c) {
  const XentPlan p = plan_xent(c.M, c.V, c.D, false);
  const uint16_t *x, *w;
  pgemm_status st = xent_operands<T>(c, p, &x, &w);
  if (st != PGEMM_OK) return st;
  float2 *part = reinterpret_cast<float2 *>(c.ws + p.part);
  float *at = reinterpret_cast<float *>(c.ws + p.at);
  FusedProduct g{};
  g.a = FusedOperand{x, nullptr, (int)p.d8, (int)c.M};
  g.b = FusedOperand{w, nullptr, (int)p.d8, (int)c.V};
  g.M = (int)c.M;
  g.N = (int)c.V;
  g.K = (int)p.d8;
  st = launch_product<T, Lay::KC, Lay::KC, false, LseEpi>(g, p.logits, LseEpi::Args{part, at, c.target}, c.stream,
                                                          c.dev);
  if (st != PGEMM_OK) return st;
  hipLaunchKernelGGL(lse_join_kernel<T>, dim3((unsigned)join_groups(c.M)), dim3(1024), 0, c.stream, part, at, c.target, c.loss,
                     c.lse, c.M, c.V, (int)p.parts, c.ignore);
  return launched();
}

template <typename T>
pgemm_status xent_backward(const XentCall &c) {
  const XentPlan p = plan_xent(c.M, c.V, c.D, true);
  const uint16_t *x, *w;
  pgemm_status st = xent_operands<T>(c, p, &x, &w);
  if (st != PGEMM_OK) return st;
  uint16_t *dz = reinterpret_cast<uint16_t *>(c.ws + p.dz);
  float *sum = reinterpret_cast<float *>(c.ws + p.sum);
  float *scale = reinterpret_cast<float *>(c.ws + p.scale);
  hipLaunchKernelGGL(loss_scale_kernel<T>, dim3(1), dim3(1024), 0, c.stream, c.dloss, c.dstep, c.target, c.M, c.ignore,
                     scale);
  st = launched();
  if (st != PGEMM_OK) return st;
  const float *unscale = scale + 1;
  for (int64_t v0 = 0; v0 < c.V; v0 += p.piece) {
    const int64_t n = c.V - v0 < p.piece ? c.V - v0 : p.piece;
    const uint16_t *wp = w + v0 * p.d8;
    FusedProduct g{};
    // dz of this piece, from its recomputed logits
    g.a = FusedOperand{x, nullptr, (int)p.d8, (int)c.M};
    g.b = FusedOperand{wp, nullptr, (int)p.d8, (int)n};
    g.M = (int)c.M;
    g.N = (int)n;
    g.K = (int)p.d8;
    st = launch_product<T, Lay::KC, Lay::KC, false, SlopeEpi>(
        g, p.logits,
        SlopeEpi::Args{dz, p.pz, c.lse_in, c.dloss, c.dstep, c.target, scale, c.ignore, v0, c.V}, c.stream, c.dev);
    if (st != PGEMM_OK) return st;
    // dW rows of this piece = dz^T x
    g.a = FusedOperand{dz, nullptr, (int)p.pz, (int)n};
    g.b = FusedOperand{x, nullptr, (int)p.d8, (int)c.D};
    g.M = (int)n;
    g.N = (int)c.D;
    g.K = (int)c.M;
    st = launch_sum<T, Lay::KR, Lay::KR>(g, p.dw,
                                         SumEpi::Args{nullptr, 0, 1, 1, {c.dw + v0 * c.D, c.D, unscale, false}}, c.ws + p.part,
                                         c.stream, c.dev);
    if (st != PGEMM_OK) return st;
    // dx += dz W
    g.a = FusedOperand{dz, nullptr, (int)p.pz, (int)c.M};
    g.b = FusedOperand{wp, nullptr, (int)p.d8, (int)c.D};
    g.M = (int)c.M;
    g.N = (int)c.D;
    g.K = (int)n;
    st = launch_sum<T, Lay::KC, Lay::KR>(
        g, shortened(p.dx, n),
        SumEpi::Args{sum, (int)p.ps, v0 == 0, v0 + n == c.V, {c.dx, c.D, unscale, false}}, c.ws + p.part, c.stream, c.dev);
    if (st != PGEMM_OK) return st;
  }
  return PGEMM_OK;
}

}  // namespace launch_detail
}  // namespace pgemm
