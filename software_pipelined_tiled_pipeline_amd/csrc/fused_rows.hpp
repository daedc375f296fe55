// Padded copies of operands whose rows do not start on 16 bytes.
#pragma once

#include "fused_launch.hpp"

namespace pgemm {

// dst[rows][pitch] = src[rows][cols], zeros from cols on (pitch a multiple of 8).
static __global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t *__restrict__ src, uint16_t *__restrict__ dst,
                                                       int64_t rows, int cols, int pitch) {
  const int per = pitch / 8;
  const int64_t total = rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    const int c = (int)(i % per) * 8;
    const uint16_t *s = src + row * cols + c;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (c + 8 <= cols) {
      v = *reinterpret_cast<const u32x4_any *>(s);
    } else {
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (c + x < cols) v[x / 2] |= (uint32_t)s[x] << (16 * (x % 2));
    }
    *reinterpret_cast<u32x4 *>(dst + row * pitch + c) = v;
  }
}

namespace launch_detail {

inline pgemm_status pad_rows(const uint16_t *src, char *dst, int64_t rows, int64_t cols, int64_t pitch,
                             hipStream_t stream) {
  if (rows == 0) return PGEMM_OK;
  hipLaunchKernelGGL(pad_rows_kernel, dim3(row_grid(rows * (pitch / 8))), dim3(256), 0, stream, src,
                     reinterpret_cast<uint16_t *>(dst), rows, (int)cols, (int)pitch);
  return launched();
}

}  // namespace launch_detail
}  // namespace pgemm
