// Launches of the 8-bit products and of the quantization of rows.
#pragma once

#include "i8.hpp"
#include "serve.hpp"

namespace pgemm {
namespace launch_detail {

template <typename T>
pgemm_status quant_rows(const uint16_t *x, int8_t *q, float *scale, int64_t M, int64_t K, hipStream_t stream) {
  if (M == 0) return PGEMM_OK;
  const int k = (int)K, width = (int)i8_width(K);
  const int64_t groups = K <= 1024 ? per(M, 4) : M;
  const dim3 grid((unsigned)(groups < 16384 ? groups : 16384));
  if (K < 8) {
    hipLaunchKernelGGL(quant_short_kernel<T>, dim3(row_grid(M)), dim3(256), 0, stream, x, q, scale, M, k);
  } else if (K <= 1024)
    hipLaunchKernelGGL((quant_rows_kernel<T, 1, 2>), grid, dim3(256), 0, stream, x, q, scale, M, k, width);
  else if (K <= 4096)
    hipLaunchKernelGGL((quant_rows_kernel<T, 4, 2>), grid, dim3(256), 0, stream, x, q, scale, M, k, width);
  else
    hipLaunchKernelGGL((quant_rows_kernel<T, 4, 4>), grid, dim3(256), 0, stream, x, q, scale, M, k, width);
  return launched();
}

template <typename T, bool GATED, int MT, int WAVES, bool XL>
pgemm_status launch_i8_few_one(const I8Args &a, hipStream_t stream, int dev) {
  static std::atomic<uint64_t> lds_set{0};
  constexpr int SUMS = (XL ? 64 : 0) + i8_sums(MT, WAVES, XL), MOST = SUMS + (XL ? kI8OwnTokens * (kI8OwnWidth + 16) : 0);
  static_assert(MOST <= 160 * 1024, "LDS of a CU");
  const int lds = SUMS + (XL ? (int)(a.M * (up_to(a.width, 256) + 16)) : 0);
  auto kern = i8_few_kernel<T, GATED, MT, WAVES, XL>;
  if (lds > 65536) {
    pgemm_status st = allow_lds(kern, MOST, dev, lds_set);
    if (st != PGEMM_OK) return st;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)per(a.N, GATED ? 16 : 32), (unsigned)per(a.M, 16 * MT)), dim3(WAVES * 64), lds,
                     stream, a);
  return launched();
}

template <typename T, bool GATED, int MT, bool XL>
pgemm_status launch_i8_waves(const I8Args &a, hipStream_t stream, int dev) {
  const int64_t groups = per(a.N, GATED ? 16 : 32) * per(a.M, 16 * MT);
  if (groups <= 512) return launch_i8_few_one<T, GATED, MT, 8, XL>(a, stream, dev);
  return launch_i8_few_one<T, GATED, MT, 4, XL>(a, stream, dev);
}

template <typename T, bool GATED>
pgemm_status launch_i8_few(const I8Args &a, bool own, hipStream_t stream, int dev) {
  if (own) return launch_i8_waves<T, GATED, 1, true>(a, stream, dev);
  if (a.M <= 16) return launch_i8_waves<T, GATED, 1, false>(a, stream, dev);
  if (a.M <= 32) return launch_i8_waves<T, GATED, 2, false>(a, stream, dev);
  return launch_i8_waves<T, GATED, 4, false>(a, stream, dev);
}

template <typename T>
pgemm_status i8_tiles(const I8Call &c, const I8Plan &p, const int8_t *q, const float *xs) {
  const int64_t units = i8_width(c.K) / 2;
  const uint16_t *w = reinterpret_cast<const uint16_t *>(c.w);
  FusedProduct g{};
  g.a = FusedOperand{reinterpret_cast<const uint16_t *>(q), nullptr, (int)units, (int)c.M};
  g.b = FusedOperand{w, c.gated ? w + c.N * units : nullptr, (int)units, (int)c.N};
  g.M = (int)c.M;
  g.N = (int)c.N;
  g.K = (int)units;
  if (c.gated)
    return launch_product<int8_t, Lay::KC, Lay::KC, true, I8GatedEpi<T>>(
        g, p.tiles, typename I8GatedEpi<T>::Args{c.out, xs, c.ws, c.act}, c.stream, c.dev);
  if (p.tiles.split == 1)
    return launch_product<int8_t, Lay::KC, Lay::KC, false, I8Epi<T>>(g, p.tiles, typename I8Epi<T>::Args{c.out, xs, c.ws},
                                                                     c.stream, c.dev);
  const int pp = (int)up_to(c.N, 4);
  int *part = reinterpret_cast<int *>(c.workspace + p.part);
  pgemm_status st = launch_product<int8_t, Lay::KC, Lay::KC, false, I8PieceEpi>(g, p.tiles, I8PieceEpi::Args{part, pp},
                                                                                c.stream, c.dev);
  if (st != PGEMM_OK) return st;
  hipLaunchKernelGGL(i8_join_kernel<T>, dim3(row_grid(c.M * (pp / 4))), dim3(256), 0, c.stream, part, p.tiles.split,
                     (int)c.M, (int)c.N, pp, xs, c.ws, c.out);
  return launched();
}

template <typename T>
pgemm_status i8_product(const I8Call &c) {
  // scales tell the kinds of tokens apart: rows of no values may have no address
  const bool quantized = c.xs != nullptr;
  const I8Plan p = plan_i8(c.M, c.N, c.K, c.gated, quantized);
  const int8_t *q = c.q;
  const float *xs = c.xs;
  if (!quantized && !p.own) {
    int8_t *to = reinterpret_cast<int8_t *>(c.workspace + p.q);
    float *scale = reinterpret_cast<float *>(c.workspace + p.s);
    pgemm_status st = quant_rows<T>(c.x, to, scale, c.M, c.K, c.stream);
    if (st != PGEMM_OK) return st;
    q = to;
    xs = scale;
  }
  if (!p.few) return i8_tiles<T>(c, p, q, xs);
  I8Args a{};
  a.x = c.x;
  a.q = q;
  a.xs = xs;
  a.w = c.w;
  a.ws = c.ws;
  a.out = c.out;
  a.M = (int)c.M;
  a.N = (int)c.N;
  a.K = (int)c.K;
  a.width = (int)i8_width(c.K);
  a.act = c.act;
  return c.gated ? launch_i8_few<T, true>(a, p.own, c.stream, c.dev) : launch_i8_few<T, false>(a, p.own, c.stream, c.dev);
}

}  // namespace launch_detail
}  // namespace pgemm
