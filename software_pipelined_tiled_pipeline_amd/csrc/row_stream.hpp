// The K loop of products with few rows (tokens) whose weights are read once:
// the 8-bit products and the mixture of experts.
//
// A wave multiplies MT blocks of 16 tokens with NT blocks of 16 weight rows,
// block of K by block of K.  Widths count units of two bytes: a 16-bit value or
// two 8-bit ones; a block is 128 of them, 256 bytes of a row, in four MFMA
// steps.  Four lanes load 64 bytes of a row, so that a load is 16 requests and
// not one a lane; the values change lanes to where the MFMAs want them, row
// l % 16, with ds_bpermute (skinny.hpp has what that is worth).  The next
// block's loads are issued step by step while this one is multiplied, also
// where the next block belongs to other rows.
//   lane l, register r of an accumulator: token 4 (l / 16) + r, weight row l % 16.
#pragma once

#include "skinny.hpp"

namespace pgemm {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// 8-bit integers: 64 of them along K a step, sums in int32 kept in a float's bits.
struct Int8Step {
  __device__ __forceinline__ static f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b),
                                                                           __builtin_bit_cast(i32x4, c), 0, 0, 0));
  }
};

// Where the tokens are: in memory like the weights; in LDS already, in whole
// blocks, where `xl` points at this lane's fragment (token l % 16, 16-byte piece
// l / 16); or in memory in fp32, to be rounded to T after a factor of their row.
enum class Tokens { Rows, Lds, Wide };

template <class F, int MT, int NT, Tokens X = Tokens::Rows, typename T = void>
struct RowStream {
  static constexpr int XD = MT == 1 && X != Tokens::Wide ? 4 : 2;  // steps that tokens are loaded ahead
  static constexpr int XP = X == Tokens::Wide ? 2 : 1;  // 16-byte pieces of a token's share

  // A block's place: where the tokens and each block of weight rows start, the
  // same for the wave; this lane's rows (row l / 4 of each block) from there,
  // below 2^31 bytes; the block of K.
  struct Place {
    const char *x, *w[NT];
    uint32_t xo[MT], wo[NT];
    float scale[MT];  // Wide: of x's rows
    int kb;
  };

  int K, full;  // units of a row; whole blocks
  int from;     // the lane its fragments come from, in bytes
  int piece;    // which 16 bytes of a step it loads
  f32x4 tot[MT][NT];
  u32x4 xr[XD][MT][XP], wr[4][NT];
  const char *xl;

  __device__ __forceinline__ void init(int lane, int units) {
    K = units;
    full = units / 128;
    from = (4 * (lane & 15) + (lane >> 4)) * 4;
    piece = lane & 3;
    clear();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int b = 0; b < NT; ++b) tot[m][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  __device__ __forceinline__ int blocks() const { return (K + 127) / 128; }

  // Eight units of a row for step s of block kb.  In the block that K ends in
  // the row's last eight, put in place when they are used.
  __device__ __forceinline__ u32x4 load(const char *base, uint32_t row, int kb, int s) const {
    if (kb < full) return load_at<u32x4_any>(base + ((int64_t)kb * 256 + s * 64), row + 16u * piece);
    const int k = kb * 128 + 32 * s + 8 * piece;
    return load_at<u32x4_any>(base, row + 2u * (k < K - 8 ? k : K - 8));
  }
  __device__ __forceinline__ u32x4 used(u32x4 v, int kb, int s) const {
    if (kb >= full) {
      const int past = kb * 128 + 32 * s + 8 * piece - (K - 8);
      v = drop_values(v, past > 0 ? past : 0);
    }
    return to_rows(v, from);
  }
  __device__ __forceinline__ void load_x(const Place &p, int slot, int s) {
    if constexpr (X == Tokens::Lds) return;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (X == Tokens::Wide) {
        const int k = p.kb * 128 + 32 * s + 8 * piece;
        const uint32_t at = p.xo[m] + 4u * (p.kb < full || k < K - 8 ? k : K - 8);
        xr[slot][m][0] = load_at<u32x4_any>(p.x, at);
        xr[slot][m][1] = load_at<u32x4_any>(p.x, at + 16u);
      } else {
        xr[slot][m][0] = load(p.x, p.xo[m], p.kb, s);
      }
    }
  }
  __device__ __forceinline__ void load_w(const Place &p, int s) {
#pragma unroll
    for (int b = 0; b < NT; ++b) wr[s][b] = load(p.w[b], p.wo[b], p.kb, s);
  }
  __device__ __forceinline__ void begin_weights(const Place &p) {
#pragma unroll
    for (int s = 0; s < 4; ++s) load_w(p, s);
  }
  __device__ __forceinline__ void begin_tokens(const Place &p) {
#pragma unroll
    for (int s = 0; s < XD; ++s) load_x(p, s, s);
  }
  __device__ __forceinline__ void begin(const Place &p) {
    begin_weights(p);
    begin_tokens(p);
  }

  // All of rows shorter than eight units, value by value (not from LDS).
  __device__ __forceinline__ void short_rows(const Place &p) {
    u32x4 x[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if constexpr (X == Tokens::Wide) {
        if (piece == 0) {
          const float *row = reinterpret_cast<const float *>(p.x + p.xo[m]);
#pragma unroll
          for (int e = 0; e < 7; ++e) {
            if (e < K) v[e / 2] |= Mfma<T>::pack4(row[e] * p.scale[m], 0.0f, 0.0f, 0.0f)[0] << (16 * (e % 2));
          }
        }
      } else {
        if (piece == 0) v = load_tail(reinterpret_cast<const uint16_t *>(p.x + p.xo[m]), 0, K);
      }
      x[m] = to_rows(v, from);
    }
#pragma unroll
    for (int b = 0; b < NT; ++b) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (piece == 0) v = load_tail(reinterpret_cast<const uint16_t *>(p.w[b] + p.wo[b]), 0, K);
      v = to_rows(v, from);
#pragma unroll
      for (int m = 0; m < MT; ++m) tot[m][b] = F::mma(x[m], v, tot[m][b]);
    }
  }

  // Block `at`, while block `next` loads (rows of eight units and more).
  template <bool MORE>
  __device__ __forceinline__ void block(const Place &at, const Place &next) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 x[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if constexpr (X == Tokens::Lds) {
          x[m] = *reinterpret_cast<const u32x4 *>(xl + at.kb * 256 + s * 64);
        } else if constexpr (X == Tokens::Wide) {
          u32x4 v;
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const f32x4 f = __builtin_bit_cast(f32x4, xr[s % XD][m][e / 4]) * at.scale[m];
            const u32x2 p = Mfma<T>::pack4(f[0], f[1], f[2], f[3]);
            v[e / 2] = p[0];
            v[e / 2 + 1] = p[1];
          }
          x[m] = used(v, at.kb, s);
        } else {
          x[m] = used(xr[s % XD][m][0], at.kb, s);
        }
      }
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const u32x4 w = used(wr[s][b], at.kb, s);
#pragma unroll
        for (int m = 0; m < MT; ++m) tot[m][b] = F::mma(x[m], w, tot[m][b]);
      }
      if (MORE) load_w(next, s);
      // the slot of step s takes step s + XD
      if (s + XD < 4)
        load_x(at, s % XD, s + XD);
      else if (MORE)
        load_x(next, s % XD, s + XD - 4);
    }
  }
};
// (Widths below eight units, in which load_tail reads a row value by value, are
// left out of the loop: its loads took 70 registers.)

// Row r of a block of rows from row0 on, the last of `rows` repeated: its
// distance from where block_start says that the block starts.
__device__ __forceinline__ const char *block_start(const void *base, int64_t row0, int64_t rows, int64_t pitch) {
  return static_cast<const char *>(base) + (row0 < rows ? row0 : rows - 1) * pitch;
}
__device__ __forceinline__ uint32_t block_row(int64_t row0, int r, int64_t rows, int64_t pitch) {
  return (uint32_t)(((row0 + r < rows ? row0 + r : rows - 1) - (row0 < rows ? row0 : rows - 1)) * pitch);
}

// Where a workgroup starts along K: rows are often a multiple of the memory
// channels' interleave apart, and all would meet on the same few.
__device__ __forceinline__ int first_turn(unsigned group, int blocks) {
  return blocks > 0 ? (int)((group * 0x9E3779B1u >> 12) % (unsigned)blocks) : 0;
}

}  // namespace pgemm
