// Launches of the products with 4-bit weights.
#pragma once

#include "fused_launch.hpp"
#include "q4.hpp"

namespace pgemm {
namespace launch_detail {

template <typename T, bool GATED, int MT, int GS, int XI, int NW, int KW, int D>
pgemm_status launch_q4_one(Q4Args a, hipStream_t stream, int dev) {
  using G = Q4Geom<T, GATED, MT, GS, XI, NW, KW, D>;
  static std::atomic<uint64_t> lds_set{0};
  constexpr int kMost = 160 * 1024;  // LDS per workgroup on gfx950
  const int64_t k = a.K < G::CB * 128 ? up_to(a.K, 128) : G::CB * 128;
  a.sp = (int)up_to(k / a.group + 2, 4) | 1;
  const int work = G::RING + G::XBYTES + G::ROWS * a.sp * 4;
  const int lds = work > G::JOIN ? work : G::JOIN;
  static_assert(G::RING + G::XBYTES + G::ROWS * (G::CB / GS * 4 + 5) * 4 <= kMost && G::JOIN <= kMost, "groups of 32 fit");
  auto kern = q4_kernel<T, GATED, MT, GS, XI, NW, KW, D>;
  if (lds > 65536) {
    pgemm_status st = allow_lds(kern, kMost, dev, lds_set);
    if (st != PGEMM_OK) return st;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)per(a.N, G::COLS), (unsigned)per(a.M, 16 * MT)), dim3(G::THREADS), lds, stream,
                     a);
  return launched();
}

// Waves along K, up to 16 tokens: so many that all workgroups together give
// each CU about sixteen.
template <typename T, bool GATED, int GS>
pgemm_status launch_q4(const Q4Args &a, hipStream_t stream, int dev) {
  const int64_t groups = per(a.N, GATED ? 16 : 32);
  if (a.M <= 4) {
    if (groups <= 256 && a.K > 8 * 128) return launch_q4_one<T, GATED, 1, GS, 1, 1, 16, 3>(a, stream, dev);
    if (groups <= 512) return launch_q4_one<T, GATED, 1, GS, 1, 1, 8, 3>(a, stream, dev);
    return launch_q4_one<T, GATED, 1, GS, 1, 1, 4, 3>(a, stream, dev);
  }
  if (a.M <= 16) {
    if (groups <= 256) return launch_q4_one<T, GATED, 1, GS, 4, 1, 8, 2>(a, stream, dev);
    return launch_q4_one<T, GATED, 1, GS, 4, 1, 4, 2>(a, stream, dev);
  }
  // Waves beside each other: a workgroup fills a CU.  Three (four) of them take
  // 1.25 (1.4) times as long as two, and need fewer rounds of 256 workgroups.
  // Groups of 64, K 4096, microseconds with two and with three (M 32 and 48) or
  // four (M 64):
  //   N      16384       24576       32000       49152
  //   M 32   17.1 19.8   29.7 20.6   29.9 36.9   43.7 38.4
  //   M 48   20.9 25.5   37.1 26.0   37.5 47.7   55.0 49.5
  //   M 64   25.6 33.9   46.3 33.9   47.0 35.6   69.0 65.2
  const int64_t blocks_m = per(a.M, 64);
  auto rounds = [&](int nw) { return per(per(groups, nw) * blocks_m, 256); };
  const int64_t two = rounds(2);
  if (a.M <= 48) {
    const bool three = rounds(3) * 5 < two * 4;
    if (a.M <= 32)
      return three ? launch_q4_one<T, GATED, 2, GS, 8, 3, 4, 2>(a, stream, dev)
                   : launch_q4_one<T, GATED, 2, GS, 8, 2, 4, 2>(a, stream, dev);
    return three ? launch_q4_one<T, GATED, 3, GS, 12, 3, 4, 2>(a, stream, dev)
                 : launch_q4_one<T, GATED, 3, GS, 12, 2, 4, 2>(a, stream, dev);
  }
  return rounds(4) * 7 < two * 5 ? launch_q4_one<T, GATED, 4, GS, 16, 4, 2, 2>(a, stream, dev)
                                 : launch_q4_one<T, GATED, 4, GS, 16, 2, 4, 2>(a, stream, dev);
}

template <typename T, bool GATED>
pgemm_status q4_groups(const Q4Args &a, hipStream_t stream, int dev) {
  if (a.group % 128 == 0) return launch_q4<T, GATED, 4>(a, stream, dev);
  if (a.group % 64 == 0) return launch_q4<T, GATED, 2>(a, stream, dev);
  return launch_q4<T, GATED, 1>(a, stream, dev);
}

template <typename T>
pgemm_status q4_product(const Q4Call &c) {
  Q4Args a{};
  a.x = c.x;
  a.q = c.q;
  a.scale = c.scale;
  a.zero = c.zero;
  a.out = c.out;
  a.M = (int)c.M;
  a.N = (int)c.N;
  a.K = (int)c.K;
  a.wb = (int)(up_to(c.K, 32) / 2);
  // one group of all of K, however much longer it is
  a.group = (int)(c.group < c.K ? c.group : up_to(c.K > 0 ? c.K : 1, 128));
  a.groups = (int)per(c.K, a.group);
  a.per32 = ((uint64_t)1 << 40) / (uint64_t)(a.group / 32) + 1;
  a.act = c.act;
  if (a.K < 8) {
    auto kern = c.gated ? q4_short_kernel<T, true> : q4_short_kernel<T, false>;
    hipLaunchKernelGGL(kern, dim3(row_grid(c.M * c.N)), dim3(256), 0, c.stream, a);
    return launched();
  }
  return c.gated ? q4_groups<T, true>(a, c.stream, c.dev) : q4_groups<T, false>(a, c.stream, c.dev);
}

}  // namespace launch_detail
}  // namespace pgemm
