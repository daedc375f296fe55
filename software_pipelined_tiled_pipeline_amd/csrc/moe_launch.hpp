// Launches of the mixture of experts.
#pragma once

#include "fused_launch.hpp"
#include "moe.hpp"

namespace pgemm {
namespace launch_detail {

constexpr int kMoeLds = 160 * 1024;  // a CU's

template <typename T, int MT, int WAVES, bool SHORT = false>
pgemm_status launch_moe_gated(const MoeArgs &a, int64_t chunks, hipStream_t stream, int dev) {
  static std::atomic<uint64_t> lds_set{0};
  constexpr int LDS = 144 + WAVES * stream_bytes(MT);
  static_assert(stream_bytes(MT) >= MT * 2048 && LDS <= 160 * 1024, "the sums take the blocks' place");
  auto kern = moe_gated_kernel<T, MT, WAVES, SHORT>;
  if (LDS > 65536) {
    pgemm_status st = allow_lds(kern, LDS, dev, lds_set);
    if (st != PGEMM_OK) return st;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)per(a.F, 16), (unsigned)a.slots, (unsigned)chunks), dim3(WAVES * 64), LDS, stream, a);
  return launched();
}

template <typename T, int MT, int WAVES, bool SHORT = false>
pgemm_status launch_moe_down(const MoeArgs &a, int64_t chunks, hipStream_t stream, int dev) {
  static std::atomic<uint64_t> lds_set{0};
  auto kern = moe_down_kernel<T, MT, WAVES, SHORT>;
  const int lds = moe_down_lds(MT, WAVES, a.M < kMoeChunk ? a.M : kMoeChunk, a.k, a.slots);
  if (lds > 65536) {
    pgemm_status st = allow_lds(kern, kMoeLds, dev, lds_set);
    if (st != PGEMM_OK) return st;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)per(a.D, kMoeColumns), (unsigned)chunks, (unsigned)a.splits), dim3(WAVES * 64), lds, stream, a);
  return launched();
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
  a.counts = reinterpret_cast<uint32_t *>(c.workspace + p.counts);
  a.lists = reinterpret_cast<uint16_t *>(c.workspace + p.lists);
  a.M = (int)c.M;
  a.E = (int)c.E;
  a.D = (int)c.D;
  a.F = (int)c.F;
  a.k = (int)c.top_k;
  a.slots = (int)p.slots;
  a.splits = (int)p.splits;
  a.groups = (int)p.groups;
  a.partial = reinterpret_cast<float *>(c.workspace + p.partial);
  a.arrived = reinterpret_cast<uint32_t *>(c.workspace + p.arrived);
  a.by_choice = p.by_choice;
  a.act = c.act;
  a.normalize = c.normalize;
  pgemm_status st;
  if (c.E <= kMoeRouteExperts && c.E * c.D <= kMoeRouteValues) {
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
  // tokens an expert has on average
  const int64_t mean = (c.M < kMoeChunkTokens ? c.M : kMoeChunkTokens) * c.top_k / c.E;
  if (c.F > 0) {
    const bool many = per(c.F, 16) * p.slots * chunks > 512;
    st = c.D < 8     ? launch_moe_gated<T, 1, 8, true>(a, chunks, c.stream, c.dev)
         : mean > 24 ? launch_moe_gated<T, 4, 4>(a, chunks, c.stream, c.dev)
         : mean > 8 ? many ? launch_moe_gated<T, 2, 4>(a, chunks, c.stream, c.dev) : launch_moe_gated<T, 2, 8>(a, chunks, c.stream, c.dev)
                    : many ? launch_moe_gated<T, 1, 4>(a, chunks, c.stream, c.dev) : launch_moe_gated<T, 1, 8>(a, chunks, c.stream, c.dev);
    if (st != PGEMM_OK) return st;
  }
  // eight waves where their rows of y find room in LDS
  const bool wide = moe_down_lds(1, 8, a.M < kMoeChunk ? a.M : kMoeChunk, a.k, a.slots) <= kMoeLds;
  return c.F < 8      ? launch_moe_down<T, 1, 4, true>(a, chunks, c.stream, c.dev)
         : mean > 24  ? launch_moe_down<T, 4, 4>(a, chunks, c.stream, c.dev)
         : mean > 8   ? launch_moe_down<T, 2, 4>(a, chunks, c.stream, c.dev)
         : wide       ? launch_moe_down<T, 1, 8>(a, chunks, c.stream, c.dev)
                      : launch_moe_down<T, 1, 4>(a, chunks, c.stream, c.dev);
}

}  // namespace launch_detail
}  // namespace pgemm
