// Launch templates of the fused products, included by the operators' own
// launch headers.
#pragma once

#include "fused.hpp"
#include "fused_epilogues.hpp"
#include "launch_impl.hpp"

namespace pgemm {
namespace launch_detail {

inline unsigned row_grid(int64_t items) {
  const int64_t b = per(items, 256);
  return (unsigned)(b < 1 ? 1 : b > 16384 ? 16384 : b);
}

template <typename T, class G, Lay LA, Lay LB, bool DUAL, class Epi>
pgemm_status launch_tiles(FusedProduct g, const typename Epi::Args &e, hipStream_t stream, int dev) {
  static std::atomic<uint64_t> lds_set{0};
  auto kern = fused_kernel<T, G, LA, LB, DUAL, Epi>;
  pgemm_status st = allow_lds(kern, G::LDS_BYTES, dev, lds_set);
  if (st != PGEMM_OK) return st;
  g.tiles_m = cdiv_i(g.M, G::BM);
  g.tiles_n = cdiv_i(g.N, DUAL ? G::BN / 2 : G::BN);
  g.group_m = kGroupM;
  hipLaunchKernelGGL(kern, dim3((unsigned)((int64_t)g.tiles_m * g.tiles_n)), dim3(G::THREADS), G::LDS_BYTES, stream, g,
                     e);
  return launched();
}

template <typename T, Lay LA, Lay LB, bool DUAL, class Epi>
pgemm_status launch_product(const FusedProduct &g, const typename Epi::Args &e, hipStream_t stream, int dev) {
  if (g.M == 0 || g.N == 0) return PGEMM_OK;
  if (large_tile(g.M, g.N, DUAL)) return launch_tiles<T, SwapGeom<2>, LA, LB, DUAL, Epi>(g, e, stream, dev);
  return launch_tiles<T, SwapGeomSmall<2>, LA, LB, DUAL, Epi>(g, e, stream, dev);
}

}  // namespace launch_detail
}  // namespace pgemm
