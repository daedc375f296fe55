// Launches of the mixture of experts.
#pragma once

#include "fused_launch.hpp"
#include "moe.hpp"

namespace pgemm {
namespace launch_detail {

template <typename T, int MT, int WAVES, bool DOWN, bool SHORT>
pgemm_status launch_moe_rows_one(const MoeArgs &a, int64_t chunks, hipStream_t stream, int dev) {
  static std::atomic<uint64_t> lds_set{0};
  constexpr int LDS = WAVES * stream_bytes(MT);
  static_assert(stream_bytes(MT) >= MT * 2048 && LDS <= 160 * 1024, "the sums take the blocks' place");
  auto kern = moe_rows_kernel<T, MT, WAVES, DOWN, SHORT>;
  if (LDS > 65536) {
    pgemm_status st = allow_lds(kern, LDS, dev, lds_set);
    if (st != PGEMM_OK) return st;
  }
  const int64_t groups = DOWN ? per(a.D, 32) : per(a.F, 16);
  hipLaunchKernelGGL(kern, dim3((unsigned)groups, (unsigned)a.slots, (unsigned)chunks), dim3(WAVES * 64), LDS, stream, a);
  return launched();
}

template <typename T, bool DOWN>
pgemm_status launch_moe_rows(const MoeArgs &a, int64_t chunks, hipStream_t stream, int dev) {
  if ((DOWN ? a.F : a.D) < 8) return launch_moe_rows_one<T, 1, 8, DOWN, true>(a, chunks, stream, dev);
  const MoeCut cut = moe_cut(a.M, a.E, a.D, a.F, a.k, DOWN);
  if (cut.blocks == 4) return launch_moe_rows_one<T, 4, 4, DOWN, false>(a, chunks, stream, dev);
  if (cut.blocks == 2)
    return cut.waves == 4 ? launch_moe_rows_one<T, 2, 4, DOWN, false>(a, chunks, stream, dev)
                          : launch_moe_rows_one<T, 2, 8, DOWN, false>(a, chunks, stream, dev);
  return cut.waves == 4 ? launch_moe_rows_one<T, 1, 4, DOWN, false>(a, chunks, stream, dev)
                        : launch_moe_rows_one<T, 1, 8, DOWN, false>(a, chunks, stream, dev);
}

template <typename T>
pgemm_status moe_layer(const MoeCall &c) {
  const MoePlan p = plan_moe(c.M, c.E, c.D, c.F, c.top_k);
  const int64_t chunks = per(c.M, kMoeChunkTokens);
  MoeArgs a{};
  a.x = c.x;
  a.router = c.router;
  a.w = c.w;
  a.down = c.down;
  a.y = c.y;
  a.experts = c.experts ? c.experts : reinterpret_cast<int32_t *>(c.workspace + p.experts);
  a.weights = c.weights ? c.weights : reinterpret_cast<float *>(c.workspace + p.weights);
  a.logits = reinterpret_cast<double *>(c.workspace + p.logits);
  a.h = c.workspace + p.h;
  a.tops = kWideHidden<T> ? reinterpret_cast<uint32_t *>(c.workspace + p.tops) : nullptr;
  a.products = reinterpret_cast<float *>(c.workspace + p.products);
  a.M = (int)c.M;
  a.E = (int)c.E;
  a.D = (int)c.D;
  a.F = (int)c.F;
  a.k = (int)c.top_k;
  a.slots = (int)p.slots;
  a.by_choice = p.by_choice;
  a.act = c.act;
  a.normalize = c.normalize;
  pgemm_status st;
  if (c.E <= kMoeRouteExperts && c.D <= kMoeRouteValues) {
    hipLaunchKernelGGL(moe_route_kernel<T>, dim3((unsigned)c.M), dim3(1024), 0, c.stream, a);
    st = launched();
  } else {
    if (c.M <= 4)
      hipLaunchKernelGGL((moe_logits_kernel<T, 1>), dim3((unsigned)c.E, (unsigned)c.M), dim3(256), 0, c.stream, a);
    else
      hipLaunchKernelGGL((moe_logits_kernel<T, 4>), dim3((unsigned)c.E, (unsigned)per(c.M, 4)), dim3(256), 0, c.stream, a);
    st = launched();
    if (st != PGEMM_OK) return st;
    auto choose = c.E <= 64 ? moe_choose_kernel<1> : c.E <= 256 ? moe_choose_kernel<4> : moe_choose_kernel<16>;
    hipLaunchKernelGGL(choose, dim3((unsigned)c.M), dim3(64), 0, c.stream, a);
    st = launched();
  }
  if (st != PGEMM_OK || c.D == 0) return st;
  if (c.F > 0) {
    st = launch_moe_rows<T, false>(a, chunks, c.stream, c.dev);
    if (st != PGEMM_OK) return st;
  }
  st = launch_moe_rows<T, true>(a, chunks, c.stream, c.dev);
  if (st != PGEMM_OK || c.top_k == 1) return st;
  hipLaunchKernelGGL(moe_sum_kernel<T>, dim3(row_grid(c.M * per(c.D, 4) * 4)), dim3(64), 0, c.stream, a);
  return launched();
}

}  // namespace launch_detail
}  // namespace pgemm
