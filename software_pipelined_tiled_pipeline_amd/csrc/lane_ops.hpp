// Sums and maxima over a wave's lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pgemm {

// A lane's value from another, zero where there is none: 0x110 + n, the lane n
// before it in its row of 16; 0x142 and 0x143, the last lane of the row before it
// or of the first half of the wave, for the rows that a mask names.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lane_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t lane_move(uint64_t v) {
  const uint32_t lo = lane_move<CTRL, ROWS>((uint32_t)v), hi = lane_move<CTRL, ROWS>((uint32_t)(v >> 32));
  return (uint64_t)hi << 32 | lo;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double lane_move(double v) {
  return __builtin_bit_cast(double, lane_move<CTRL, ROWS>(__builtin_bit_cast(uint64_t, v)));
}
__device__ __forceinline__ uint64_t read_lane(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}
__device__ __forceinline__ double read_lane(double v, int lane) {
  return __builtin_bit_cast(double, read_lane(__builtin_bit_cast(uint64_t, v), lane));
}

// Sums over the lanes up to each one.
template <typename U>
__device__ __forceinline__ U wave_scan(U v) {
  v += lane_move<0x111, 0xf>(v);
  v += lane_move<0x112, 0xf>(v);
  v += lane_move<0x114, 0xf>(v);
  v += lane_move<0x118, 0xf>(v);
  v += lane_move<0x142, 0xa>(v);
  v += lane_move<0x143, 0xc>(v);
  return v;
}

// The largest of all lanes'.
__device__ __forceinline__ uint64_t wave_most(uint64_t v) {
  auto more = [](uint64_t a, uint64_t b) { return a > b ? a : b; };
  v = more(v, lane_move<0x111, 0xf>(v));
  v = more(v, lane_move<0x112, 0xf>(v));
  v = more(v, lane_move<0x114, 0xf>(v));
  v = more(v, lane_move<0x118, 0xf>(v));
  v = more(v, lane_move<0x142, 0xa>(v));
  v = more(v, lane_move<0x143, 0xc>(v));
  return read_lane(v, 63);
}

}  // namespace pgemm
