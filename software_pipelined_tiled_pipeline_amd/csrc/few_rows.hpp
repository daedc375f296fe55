// Parts that the products with few rows share: MFMA fragments, 4-bit weights,
// loads at the end of a row, and the join of a workgroup's waves.
#pragma once

#include "fused_epilogues.hpp"

namespace pgemm {

// A constant the compiler knows nothing of, in a scalar or a vector register:
// (v & mask) | bits with one of each is one instruction, with two literals two.
__device__ __forceinline__ uint32_t scalar_constant(uint32_t v) {
  asm("" : "+s"(v));
  return v;
}
__device__ __forceinline__ uint32_t vector_constant(uint32_t v) {
  asm("" : "+v"(v));
  return v;
}

// MFMA fragments of eight values, and how eight 4-bit weights (a dword, the
// first in the lowest bits) become one.  A pair of weights j and j + 4 is cut
// out of both halves of the dword at once and put into the fraction of a power
// of two; the fragment's order is 0 4 1 5 2 6 3 7.  (Integers made floating point in
// this way: Y. J. Kim et al., "Who Says Elephants Can't Run: Bringing Large Scale
// MoE Models into Cloud Scale Production", 2022.)
template <typename T>
struct Frag8;
template <>
struct Frag8<_Float16> {
  __device__ __forceinline__ static f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  // 1024 + q and 1024 + 16 q become q - zero, exactly: integers of at most 1279
  static constexpr bool kExactZero = true;
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  // a scale and a zero point in a dword: the scale's bits above -1024 - zero
  __device__ __forceinline__ static uint32_t pack(uint16_t scale, uint32_t zero) {
    return (uint32_t)scale << 16 | __builtin_bit_cast(uint16_t, (_Float16)(-1024.0f - (float)zero));
  }
  struct Zero {
    f16x2 low, high;
    __device__ __forceinline__ void set(uint32_t packed) {
      const _Float16 z = __builtin_bit_cast(_Float16, (uint16_t)packed);
      const _Float16 h = z + (_Float16)960.0f;  // -64 - zero
      low = f16x2{z, z};
      high = f16x2{h, h};
    }
  };
  struct Bits {
    uint32_t low = scalar_constant(0x000F000Fu), high = scalar_constant(0x00F000F0u), one = vector_constant(0x64006400u);
  };
  __device__ __forceinline__ static u32x4 weights(uint32_t v, const Zero &z, const Bits &k) {
    const f16x2 part = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t u = v >> 8;
    const f16x2 a = __builtin_bit_cast(f16x2, (v & k.low) | k.one) + z.low;
    const f16x2 b = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (v & k.high) | k.one), part, z.high);
    const f16x2 c = __builtin_bit_cast(f16x2, (u & k.low) | k.one) + z.low;
    const f16x2 d = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (u & k.high) | k.one), part, z.high);
    return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                 __builtin_bit_cast(uint32_t, d)};
  }
};
template <>
struct Frag8<__bf16> {
  __device__ __forceinline__ static f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  // there is no packed bf16 addition: the weights stay 16 + q, and 16 + zero
  // times the sum of x is taken off the product
  static constexpr bool kExactZero = false;
  __device__ __forceinline__ static u32x4 ones(bool in) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = vector_constant(in ? 0x3F803F80u : 0u);
    return v;
  }
  // a scale and a zero point in a dword: the scale's bits above the zero point
  __device__ __forceinline__ static uint32_t pack(uint16_t scale, uint32_t zero) { return (uint32_t)scale << 16 | zero; }
  // what a unit of x adds too much, negative (exact: 8 bits times 9)
  __device__ __forceinline__ static float excess(uint32_t packed) {
    return widen<__bf16>((uint16_t)(packed >> 16)) * (-16.0f - (float)(packed & 0xffu));
  }
  struct Zero {
    __device__ __forceinline__ void set(uint32_t) {}
  };
  struct Bits {
    uint32_t mask = scalar_constant(0x00780078u), one = vector_constant(0x41804180u);
  };
  __device__ __forceinline__ static u32x4 weights(uint32_t v, const Zero &, const Bits &k) {
    return u32x4{((v << 3) & k.mask) | k.one, ((v >> 1) & k.mask) | k.one, ((v >> 5) & k.mask) | k.one,
                 ((v >> 9) & k.mask) | k.one};
  }
};

// x in the order of Frag8::weights
__device__ __forceinline__ u32x4 weight_order(u32x4 v) {
  u32x4 o;
  o[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
  o[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
  o[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
  o[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
  return o;
}

typedef uint64_t __attribute__((aligned(2))) u64_any;
typedef uint32_t __attribute__((aligned(1))) u32_any;

template <typename U>
__device__ __forceinline__ U load_at(const void *base, uint32_t off) {
  return *reinterpret_cast<const U *>(static_cast<const char *>(base) + off);
}

// Sixteen bytes shifted down by whole values, zeros coming in.
__device__ __forceinline__ u32x4 drop_values(u32x4 v, int values) {
  const int bits = 16 * values;
  const uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
  uint64_t l, h;
  if (bits == 0) {
    l = lo;
    h = hi;
  } else if (bits < 64) {
    l = lo >> bits | hi << (64 - bits);
    h = hi >> bits;
  } else {
    l = bits < 128 ? hi >> (bits - 64) : 0;
    h = 0;
  }
  return u32x4{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
}

// Eight values of a row of K from k on, zeros from K on.  Reads inside the row
// alone: the row's last eight values, shifted, where fewer are left.
__device__ __forceinline__ u32x4 load_tail(const uint16_t *row, int k, int K) {
  if (K < 8) {
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t one = row[k + e < K ? k + e : K - 1];
      v[e / 2] |= (k + e < K ? one : 0u) << (16 * (e % 2));
    }
    return v;
  }
  const int at = k < K - 8 ? k : K - 8;
  return drop_values(*reinterpret_cast<const u32x4_any *>(row + at), k - at);
}

// Adds the sums of the `parts` waves that worked on the same output up, and
// stores it: row r of an accumulator's lane l is token 4 (l / 16) + r, and its
// column l % 16.  `sums` holds [parts][MT * NT * 4][64] floats; the block's
// waves `first`, first + step, .. take its values in turn.  `checked` gets each
// sum with its token and weight row.
template <typename T, bool GATED, int MT, int NT, typename Checked>
__device__ __forceinline__ void join_and_store(const float *sums, int parts, int64_t part_stride, int first, int step,
                                               int lane, int act, uint16_t *out, int M, int N, int m0, int n0,
                                               Checked checked) {
  constexpr int OB = GATED ? NT / 2 : NT;
  const int c = lane & 15, q = lane >> 4;
  auto joined = [&](int m, int b, int r) {
    float v = 0.0f;
    for (int w = 0; w < parts; ++w) v += sums[w * part_stride + ((m * NT + b) * 4 + r) * 64 + lane];
    return v;
  };
  for (int i = first; i < MT * OB * 4; i += step) {
    const int m = i / (OB * 4), b = i / 4 % OB, r = i % 4;
    const int row = m0 + 16 * m + 4 * q + r, col = n0 + 16 * b + c;
    if (m0 + 16 * m + r >= M) continue;  // no token in any lane
    float v = joined(m, GATED ? 2 * b : b, r), u = GATED ? joined(m, 2 * b + 1, r) : 0.0f;
    if (row < M && col < N) {
      v = checked(v, row, col);
      if constexpr (GATED) v = activate(act, v) * checked(u, row, (int64_t)col + N);
      const T t = (T)v;
      out[(int64_t)row * N + col] = __builtin_bit_cast(uint16_t, t);
    }
  }
}

}  // namespace pgemm
