// Launch templates of the fused products, included by the operators' own
// launch headers.
#pragma once

#include "fused.hpp"
#include "fused_epilogues.hpp"
#include "launch_impl.hpp"

namespace pgemm {

// Adds the pieces' partial sums up in the order of K, four columns a thread,
// and does with the sum what SumEpi does with a product's.  Bound by memory:
// four pieces of 1021 x 1000 take 5.5 us, 3.3 TB/s and the launch.
template <typename T>
__global__ void __launch_bounds__(256) join_pieces_kernel(const float *__restrict__ part, int pieces, int M, int N, int pp,
                                                          SumEpi::Args e) {
  const int per_row = pp / 4;
  const int64_t total = (int64_t)M * per_row, stride = (int64_t)M * pp;
  const float k = e.last && e.out.scale ? *e.out.scale : 1.0f;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_row;
    const int col = (int)(i % per_row) * 4;
    const float *p = part + i * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = 0; s < pieces; ++s) v += *reinterpret_cast<const f32x4 *>(p + s * stride);
    if (!e.first) v += *reinterpret_cast<const f32x4 *>(e.sum + row * e.ps + col);
    if (!e.last) {
      *reinterpret_cast<f32x4 *>(e.sum + row * e.ps + col) = v;
      continue;
    }
    const u32x2 r = Mfma<T>::pack4(v[0] * k, v[1] * k, v[2] * k, v[3] * k);
    uint16_t *dst = e.out.out + row * e.out.po + col;
    if (col + 4 <= N) {
      *reinterpret_cast<u32x2_any *>(dst) = r;
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (col + x < N) dst[x] = (uint16_t)(r[x / 2] >> (16 * (x % 2)));
    }
  }
}

namespace launch_detail {

inline unsigned row_grid(int64_t items) {
  const int64_t b = per(items, 256);
  return (unsigned)(b < 1 ? 1 : b > 16384 ? 16384 : b);
}

// Tiles of rows [g.m_base, m_end) and columns [g.n_base, n_end).
template <typename T, class G, Lay LA, Lay LB, bool DUAL, class Epi>
pgemm_status launch_tiles(FusedProduct g, int64_t m_end, int64_t n_end, int split, int64_t k_chunk,
                          const typename Epi::Args &e, hipStream_t stream, int dev) {
  static std::atomic<uint64_t> lds_set{0};
  auto kern = fused_kernel<T, G, LA, LB, DUAL, Epi>;
  pgemm_status st = allow_lds(kern, G::LDS_BYTES, dev, lds_set);
  if (st != PGEMM_OK) return st;
  g.tiles_m = cdiv_i((int)(m_end - g.m_base), G::BM);
  g.tiles_n = cdiv_i((int)(n_end - g.n_base), DUAL ? G::BN / 2 : G::BN);
  g.group_m = kGroupM;
  g.k_chunk = (int)k_chunk;
  hipLaunchKernelGGL(kern, dim3((unsigned)((int64_t)g.tiles_m * g.tiles_n * split)), dim3(G::THREADS), G::LDS_BYTES,
                     stream, g, e);
  return launched();
}

template <typename T, Lay LA, Lay LB, bool DUAL, class Epi>
pgemm_status launch_small(const FusedProduct &g, const Tiling &t, const typename Epi::Args &e, hipStream_t stream, int dev) {
  if (t.deep) return launch_tiles<T, SwapGeomSmall<4>, LA, LB, DUAL, Epi>(g, g.M, g.N, t.split, t.k_chunk, e, stream, dev);
  return launch_tiles<T, SwapGeomSmall<2>, LA, LB, DUAL, Epi>(g, g.M, g.N, t.split, t.k_chunk, e, stream, dev);
}

// What an epilogue needs of a cut product's second launch: statistics go after
// those of the first one's tiles.
template <class Args>
Args second_launch(const Args &e, const FusedProduct &, const Tiling &) {
  return e;
}
inline LseEpi::Args second_launch(LseEpi::Args e, const FusedProduct &g, const Tiling &t) {
  e.part += t.cut_n / 256 * 2 * g.M;
  return e;
}

template <typename T, Lay LA, Lay LB, bool DUAL, class Epi>
pgemm_status launch_product(FusedProduct g, const Tiling &t, const typename Epi::Args &e, hipStream_t stream, int dev) {
  if (g.M == 0 || g.N == 0) return PGEMM_OK;
  if (!t.large) return launch_small<T, LA, LB, DUAL, Epi>(g, t, e, stream, dev);
  const int64_t m = t.cut_m && t.cut_m < g.M ? t.cut_m : g.M, n = t.cut_n && t.cut_n < g.N ? t.cut_n : g.N;
  pgemm_status st = launch_tiles<T, SwapGeom<2>, LA, LB, DUAL, Epi>(g, m, n, t.split, t.k_chunk, e, stream, dev);
  if (st != PGEMM_OK || (m == g.M && n == g.N)) return st;
  g.m_base = m < g.M ? (int)m : 0;
  g.n_base = n < g.N ? (int)n : 0;
  return launch_small<T, LA, LB, DUAL, Epi>(g, t, second_launch(e, g, t), stream, dev);
}

// out = round(scale * (A B + what is in sum)): one product, or one of a series
// (SumEpi), in pieces of K as `t` says; `part` holds their partial sums.
template <typename T, Lay LA, Lay LB>
pgemm_status launch_sum(const FusedProduct &g, const Tiling &t, const SumEpi::Args &e, char *part, hipStream_t stream,
                        int dev) {
  if (g.M == 0 || g.N == 0) return PGEMM_OK;
  if (t.split > 1) {
    const int pp = (int)up_to(g.N, 4);
    float *sums = reinterpret_cast<float *>(part);
    pgemm_status st = launch_product<T, LA, LB, false, PieceEpi>(
        g, t, PieceEpi::Args{sums, pp, e.out.seeded ? e.out.out : nullptr, e.out.po}, stream, dev);
    if (st != PGEMM_OK) return st;
    hipLaunchKernelGGL(join_pieces_kernel<T>, dim3(row_grid((int64_t)g.M * (pp / 4))), dim3(256), 0, stream, sums, t.split,
                       g.M, g.N, pp, e);
    return launched();
  }
  if (e.first && e.last) return launch_product<T, LA, LB, false, StoreEpi>(g, t, e.out, stream, dev);
  return launch_product<T, LA, LB, false, SumEpi>(g, t, e, stream, dev);
}

}  // namespace launch_detail
}  // namespace pgemm
