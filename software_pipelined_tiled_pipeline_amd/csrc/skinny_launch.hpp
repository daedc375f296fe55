// Launch templates of the products with few rows.
#pragma once

#include "fused_launch.hpp"
#include "skinny.hpp"

namespace pgemm {
namespace launch_detail {

template <typename T, bool GATED, int MT, int NT, int WAVES>
pgemm_status launch_skinny_one(const SkinnyArgs &a, hipStream_t stream, int dev) {
  static std::atomic<uint64_t> lds_set{0};
  constexpr int LDS = WAVES * MT * NT * 4 * 64 * 4;
  auto kern = skinny_kernel<T, GATED, MT, NT, WAVES>;
  if (LDS > 65536) {
    pgemm_status st = allow_lds(kern, LDS, dev, lds_set);
    if (st != PGEMM_OK) return st;
  }
  constexpr int cols = (GATED ? NT / 2 : NT) * 16;
  hipLaunchKernelGGL(kern, dim3((unsigned)per(a.N, cols), (unsigned)per(a.M, 16 * MT)), dim3(WAVES * 64), LDS, stream,
                     a);
  return launched();
}

// Waves along K: so many that all workgroups together give each CU about
// sixteen.
template <typename T, bool GATED, int MT>
pgemm_status launch_skinny_waves(const SkinnyArgs &a, hipStream_t stream, int dev) {
  const int64_t groups = per(a.N, GATED ? 16 : 32) * per(a.M, 16 * MT);
  if (groups <= 512) return launch_skinny_one<T, GATED, MT, 2, 8>(a, stream, dev);
  return launch_skinny_one<T, GATED, MT, 2, 4>(a, stream, dev);
}

// Token blocks of 16 a workgroup takes: as many as there are, up to four.
template <typename T, bool GATED>
pgemm_status launch_skinny(const SkinnyArgs &a, hipStream_t stream, int dev) {
  if (a.M <= 16) return launch_skinny_waves<T, GATED, 1>(a, stream, dev);
  if (a.M <= 32) return launch_skinny_waves<T, GATED, 2>(a, stream, dev);
  return launch_skinny_waves<T, GATED, 4>(a, stream, dev);
}

}  // namespace launch_detail
}  // namespace pgemm
