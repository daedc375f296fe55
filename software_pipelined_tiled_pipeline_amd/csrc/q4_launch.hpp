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

// Waves along K, with up to 4 tokens: so many that all workgroups together give each CU
// about sixteen.  With 5 to 16 tokens a workgroup has eight waves up to 256
// workgroups and four beyond, so that a CU has 4 to 8 waves between 257 and 512 of them.
template <typename T, bool GATED, int GS>
pgemm_status launch_q4(const Q4Args &a, hipStream_t stream, int dev) {
  const int64_t groups = per(a.N, GATED ? 16 : 32);
  if (a.M <= 4) {
    if (groups <= 256 && a.K > 8 * 128) return launch_q4_one<T, GATED, 1, GS, 1, 1, 16, 3>(a, stream, dev);
    if (groups <= 512) return launch_q4_one<T, GATED, 1, GS, 1, 1, 8, 3>(a, stream, dev);
    return launch_q4_one<T, GATED, 1, GS, 1, 1, 4, 3>(a, stream, dev);
  }
  // More than 16 tokens: 16 of them a workgroup, which reads weights again for
  // every 16 but has no wave wait for another, or up to 64 shared by two, three
  // or four waves beside each other, whose workgroup fills a CU.  The costs are
  // of a round of 256 workgroups, in tenths of a microsecond, measured at K 4096 in
  // groups of 64 in bf16; they decide for every K, group and type.  Microseconds
  // there with 16 tokens a workgroup, two waves, and three (M 32 and 48) or four (M 64):
  //   N          4480             12288            16384            24576            49152
  //   M 32   10.3 14.8 18.4   14.9 16.1 19.6   19.1 16.9 19.8   26.9 29.7 20.6   50.7 43.7 38.4
  //   M 48   10.6 18.8 23.9   22.0 20.4 24.8   27.7 21.3 25.5   39.6 37.1 26.0   72.6 55.0 49.5
  //   M 64   14.8 22.9 32.2   25.8 25.1 34.0   34.3 26.1 33.9   49.4 46.3 33.9   95.4 69.0 65.2
  const int blocks = a.M <= 32 ? 2 : a.M <= 48 ? 3 : 4;  // of 16 tokens, beside two waves or more
  const int64_t blocks_m = per(a.M, 64);
  auto rounds = [&](int nw) { return per(per(groups, nw) * blocks_m, 256); };
  const int64_t one = 25 + 42 * per(groups * per(a.M, 16), 256);
  const int64_t two = (blocks == 2 ? 155 : blocks == 3 ? 195 : 240) * rounds(2);
  const int64_t more = blocks == 4 ? 340 * rounds(4) : (blocks == 2 ? 200 : 255) * rounds(3);
  if (a.M <= 16 || (one < two && one < more)) {
    if (groups <= 256) return launch_q4_one<T, GATED, 1, GS, 4, 1, 8, 2>(a, stream, dev);
    return launch_q4_one<T, GATED, 1, GS, 4, 1, 4, 2>(a, stream, dev);
  }
  if (blocks == 2)
    return two <= more ? launch_q4_one<T, GATED, 2, GS, 8, 2, 4, 2>(a, stream, dev)
                       : launch_q4_one<T, GATED, 2, GS, 8, 3, 4, 2>(a, stream, dev);
  if (blocks == 3)
    return two <= more ? launch_q4_one<T, GATED, 3, GS, 12, 2, 4, 2>(a, stream, dev)
                       : launch_q4_one<T, GATED, 3, GS, 12, 3, 4, 2>(a, stream, dev);
  return two <= more ? launch_q4_one<T, GATED, 4, GS, 16, 2, 4, 2>(a, stream, dev)
                     : launch_q4_one<T, GATED, 4, GS, 16, 4, 2, 2>(a, stream, dev);
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
