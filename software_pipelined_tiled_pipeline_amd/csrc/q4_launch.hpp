// Launches of the products with 4-bit weights.
#pragma once

#include "skinny_launch.hpp"

namespace pgemm {
namespace launch_detail {

template <typename T, bool GATED>
pgemm_status q4_groups(const SkinnyArgs &a, hipStream_t stream, int dev) {
  if (a.group % 128 == 0) return launch_skinny<T, true, GATED, 4>(a, stream, dev);
  if (a.group % 64 == 0) return launch_skinny<T, true, GATED, 2>(a, stream, dev);
  return launch_skinny<T, true, GATED, 1>(a, stream, dev);
}

template <typename T>
pgemm_status q4_product(const Q4Call &c) {
  SkinnyArgs a{};
  a.x = c.x;
  a.w = c.q;
  a.scale = c.scale;
  a.zero = c.zero;
  a.out = c.out;
  a.M = (int)c.M;
  a.N = (int)c.N;
  a.K = (int)c.K;
  a.wb = up_to(c.K, 32) / 2;
  a.group = c.group;
  a.groups = (int)per(c.K, c.group);
  a.act = c.act;
  return c.gated ? q4_groups<T, true>(a, c.stream, c.dev) : q4_groups<T, false>(a, c.stream, c.dev);
}

}  // namespace launch_detail
}  // namespace pgemm
