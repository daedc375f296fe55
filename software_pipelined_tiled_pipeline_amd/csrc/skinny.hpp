// Products with few rows (tokens): out = x W^T, or the gated block
// act(x Wg^T) * (x Wu^T), bound by reading the weights once.
//
// A workgroup owns NT blocks of 16 weight rows and all of K; its waves take
// blocks of 128 k in turn, so that a weight row's loads are in flight on
// several waves at once, and add their sums up in LDS at the end.  There is
// no LDS on the weights' way: a lane loads 16 bytes of row l % 16 and the
// values go into v_mfma_f32_16x16x32 as they are, with the tokens (up to 16,
// rows past M as zeros) as the other operand:
//   lane l, register r of an accumulator: token 4 (l / 16) + r, weight row l % 16.
//
// Weights are 16-bit (W16) or 4-bit with a scale per group of a row (W4).
#pragma once

#include "fused_epilogues.hpp"

namespace pgemm {

struct SkinnyArgs {
  const uint16_t *x;  // [M][K]
  const void *w;      // W16: [rows][K]; W4: [rows][wb] bytes
  const uint16_t *scale;
  const uint8_t *zero;  // W4: [rows][groups]; zero may be null (8)
  uint16_t *out;        // [M][N]
  int M, N, K;          // N output columns; the gated block has 2 N weight rows
  int64_t wb;           // bytes of a weight row
  int group, groups;    // W4
  int act;
};

template <typename T>
struct Frag8;
template <>
struct Frag8<_Float16> {
  typedef f16x8 type;
  __device__ __forceinline__ static f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static constexpr uint32_t kOne2 = 0x3C003C00u;
  // Pairs {16 + nibble j, 16 + nibble j + 4} of a dword: the nibble goes to
  // the top of 16's fraction bits.
  __device__ __forceinline__ static u32x4 nibbles(uint32_t v) {
    constexpr uint32_t m = 0x03C003C0u, one = 0x4C004C00u;
    return u32x4{((v << 6) & m) | one, ((v << 2) & m) | one, ((v >> 2) & m) | one, ((v >> 6) & m) | one};
  }
};
template <>
struct Frag8<__bf16> {
  typedef bf16x8 type;
  __device__ __forceinline__ static f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static constexpr uint32_t kOne2 = 0x3F803F80u;
  __device__ __forceinline__ static u32x4 nibbles(uint32_t v) {
    constexpr uint32_t m = 0x00780078u, one = 0x41804180u;
    return u32x4{((v << 3) & m) | one, ((v >> 1) & m) | one, ((v >> 5) & m) | one, ((v >> 9) & m) | one};
  }
};

// Eight values of row `row` of src[rows][cols] from column k on; zeros outside.
__device__ __forceinline__ u32x4 load8(const uint16_t *src, int row, int rows, int k, int cols) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (row < rows && k < cols) {
    const uint16_t *p = src + (int64_t)row * cols + k;
    if (k + 8 <= cols) {
      v = *reinterpret_cast<const u32x4_any *>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < cols) v[e / 2] |= (uint32_t)p[e] << (16 * (e % 2));
    }
  }
  return v;
}

// The order in which Frag8::nibbles leaves eight weights: 0 4 1 5 2 6 3 7.
__device__ __forceinline__ u32x4 nibble_order(u32x4 v) {
  u32x4 o;
  o[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
  o[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
  o[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
  o[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
  return o;
}

// 4 x 4 transposition between a lane's four dwords and the four rows of 16
// lanes: a lane in row q of the result holds, in dword s, dword q of row s.
__device__ __forceinline__ u32x4 rows_to_steps(u32x4 v) {
  auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

// GS: k32 steps that share a scale before the sums are scaled (4-bit only):
// 4 when the group is a multiple of 128, 2 of 64, else 1.
template <typename T, bool W4, bool GATED, int MT, int NT, int GS, int WAVES>
__global__ void __launch_bounds__(WAVES * 64) skinny_kernel(SkinnyArgs a) {
  static_assert(!GATED || NT % 2 == 0, "gate and up blocks come in pairs");
  using F = Frag8<T>;
  extern __shared__ __attribute__((aligned(16))) float sums[];  // [WAVES][MT * NT * 4][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, q = lane >> 4;
  constexpr int OB = GATED ? NT / 2 : NT;  // output blocks of 16 columns
  const int n0 = blockIdx.x * OB * 16, m0 = blockIdx.y * MT * 16;

  // this lane's weight row in each block (a row past the end repeats the last
  // one; its column is not stored)
  int64_t wrow[NT];
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    int n = n0 + (GATED ? b / 2 : b) * 16 + c;
    n = n < a.N ? n : a.N - 1;
    wrow[b] = GATED && (b & 1) ? n + a.N : n;
  }
  f32x4 tot[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int b = 0; b < NT; ++b) tot[m][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int blocks = (a.K + 127) / 128;
  for (int kb = wave; kb < blocks; kb += WAVES) {
    const int k0 = kb * 128;
    if constexpr (W4) {
      u32x4 w[NT];
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        // bytes past the row's end meet x = 0
        const int64_t off = (int64_t)kb * 64 + q * 16;
        w[b] = off < a.wb ? *reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.w) + wrow[b] * a.wb + off)
                          : u32x4{0u, 0u, 0u, 0u};
        w[b] = rows_to_steps(w[b]);
      }
#pragma unroll
      for (int s0 = 0; s0 < 4; s0 += GS) {
        f32x4 acc[MT][NT], xs[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          xs[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int b = 0; b < NT; ++b) acc[m][b] = xs[m];
        }
#pragma unroll
        for (int s = s0; s < s0 + GS; ++s) {
          u32x4 x[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            x[m] = nibble_order(load8(a.x, m0 + 16 * m + c, a.M, k0 + 32 * s + 8 * q, a.K));
            // the weights carry 16 too much: the sum of x takes it out again
            xs[m] = F::mma(x[m], u32x4{F::kOne2, F::kOne2, F::kOne2, F::kOne2}, xs[m]);
          }
#pragma unroll
          for (int b = 0; b < NT; ++b) {
            const u32x4 f = F::nibbles(w[b][s]);
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[m][b] = F::mma(x[m], f, acc[m][b]);
          }
        }
        int gi = (k0 + 32 * s0) / a.group;
        gi = gi < a.groups ? gi : a.groups - 1;
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          const int64_t at = wrow[b] * a.groups + gi;
          const float sc = widen<T>(a.scale[at]);
          const float z = 16.0f + (a.zero ? (float)a.zero[at] : 8.0f);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) tot[m][b][r] += sc * (acc[m][b][r] - z * xs[m][r]);
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        u32x4 x[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = load8(a.x, m0 + 16 * m + c, a.M, k0 + 32 * s + 8 * q, a.K);
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          // 64-bit row offsets: load8 takes the row's own start
          const u32x4 f = load8(static_cast<const uint16_t *>(a.w) + wrow[b] * a.K, 0, 1, k0 + 32 * s + 8 * q, a.K);
#pragma unroll
          for (int m = 0; m < MT; ++m) tot[m][b] = F::mma(x[m], f, tot[m][b]);
        }
      }
    }
  }
  constexpr int VALS = MT * NT * 4;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[(wave * VALS + (m * NT + b) * 4 + r) * 64 + lane] = tot[m][b][r];
  __syncthreads();
  auto joined = [&](int m, int b, int r) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += sums[(w * VALS + (m * NT + b) * 4 + r) * 64 + lane];
    return v;
  };
  for (int i = wave; i < MT * OB * 4; i += WAVES) {
    const int m = i / (OB * 4), b = i / 4 % OB, r = i % 4;
    const int row = m0 + 16 * m + 4 * q + r, col = n0 + 16 * b + c;
    float v;
    if constexpr (GATED)
      v = activate(a.act, joined(m, 2 * b, r)) * joined(m, 2 * b + 1, r);
    else
      v = joined(m, b, r);
    if (row < a.M && col < a.N) {
      const T t = (T)v;
      a.out[(int64_t)row * a.N + col] = __builtin_bit_cast(uint16_t, t);
    }
  }
}

}  // namespace pgemm
