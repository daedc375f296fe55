// What the C entry points of the fused and serving operators check their
// arguments with, and the device and workspace of a checked call.
#pragma once

#include "fused.hpp"

namespace pgemm {
namespace api {

// Below 2^31, and so are the rows of the last tile that lie past a matrix's end.
constexpr int64_t kMaxDim = ((int64_t)1 << 31) - 255;
// Widths that are a row pitch inside a product (D, 2 F, K): a tile's rows or
// its 64 K rows then stay below 2^31 bytes, the reach of a buffer offset.
constexpr int64_t kMaxPitch = (int64_t)1 << 22;

inline bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
inline bool missing(const void *p, int64_t n) { return n > 0 && !p; }
inline bool dim(int64_t n) { return n >= 0 && n < kMaxDim; }
inline bool pitch(int64_t n) { return n >= 0 && n <= kMaxPitch; }
// a product's grid, in work-items, fits a dispatch in large tiles of 256 x 128
// columns or more (plan_tiles takes no other cut that does not, and the other
// kernels' grids are bounded where they are launched)
inline bool grid_fits(int64_t M, int64_t N) { return per(M, 256) * per(N, 128) * 256 < kMaxWorkItems; }
inline bool act_ok(int act) { return act == PGEMM_ACT_SILU || act == PGEMM_ACT_GELU; }

// Device and workspace of a checked call.
struct Site {
  int dev = 0;
  char *ws = nullptr;
  std::unique_lock<std::mutex> lock;
  pgemm_status open(void *stream, int64_t bytes) {
    pgemm_status st = checked_device(&dev);
    if (st != PGEMM_OK || bytes == 0) return st;
    return stream_workspace(dev, stream, bytes, &lock, &ws);
  }
};

}  // namespace api
}  // namespace pgemm
