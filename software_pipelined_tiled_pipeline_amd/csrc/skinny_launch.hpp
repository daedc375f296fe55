// Launch templates of the gated block with few rows.
#pragma once

#include "fused_launch.hpp"
#include "skinny.hpp"

namespace pgemm {
namespace launch_detail {

template <typename T, int MT, int WAVES>
pgemm_status launch_skinny_one(const SkinnyArgs &a, hipStream_t stream) {
  constexpr int LDS = WAVES * MT * SkinnyRun<T, MT>::NT * 4 * 64 * 4;
  static_assert(LDS <= 65536, "what a kernel may use without asking");
  auto kern = skinny_kernel<T, MT, WAVES>;
  hipLaunchKernelGGL(kern, dim3((unsigned)per(a.N, 16), (unsigned)per(a.M, 16 * MT)), dim3(WAVES * 64), LDS, stream, a);
  return launched();
}

// Waves along K: so many that all workgroups together give each CU about
// sixteen.
template <typename T, int MT>
pgemm_status launch_skinny_waves(const SkinnyArgs &a, hipStream_t stream) {
  const int64_t groups = per(a.N, 16) * per(a.M, 16 * MT);
  if (groups <= 512) return launch_skinny_one<T, MT, 8>(a, stream);
  return launch_skinny_one<T, MT, 4>(a, stream);
}

// Token blocks of 16 a workgroup takes: as many as there are, up to four.
template <typename T>
pgemm_status launch_skinny(const SkinnyArgs &a, hipStream_t stream) {
  if (a.M <= 16) return launch_skinny_waves<T, 1>(a, stream);
  if (a.M <= 32) return launch_skinny_waves<T, 2>(a, stream);
  return launch_skinny_waves<T, 4>(a, stream);
}

}  // namespace launch_detail
}  // namespace pgemm
