// The K loop of products with few rows (tokens) whose weights are read once:
// the 8-bit products and the mixture of experts.
//
// A wave multiplies MT blocks of 16 tokens with NT blocks of 16 weight rows,
// block of K by block of K.  Widths count units of two bytes: a 16-bit value or
// two 8-bit ones; a block is 128 of them, 256 bytes of a row, in four MFMA
// steps.  Sixteen lanes load a row's 256 bytes, four rows a load, so that rows
// that start on no cache line cost few lines twice; the block goes through 4 KiB
// of LDS of the wave's own to where the MFMAs want it, row l % 16.  (With four
// lanes to 64 bytes of a row, and the lanes changed by ds_bpermute as in
// skinny.hpp, the gated blocks of 60 experts of 2050 x 1001 values took 109 us
// instead of 88 for 37 tokens' four choices.)  The next block's loads are on the way
// while this one is multiplied.
//   lane l, register r of an accumulator: row 4 (l / 16) + r of the tokens, weight row l % 16.
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
// l / 16); or in memory in fp32, where eight of them are a block: a row's values
// times its factor are rounded to T for row 2 i of the block, and what that leaves
// for row 2 i + 1.
enum class Tokens { Rows, Lds, Wide };

constexpr int kBlockBytes = 4096;  // of 16 rows
// What rounding to T leaves of a number; nothing of an infinite one or a NaN.
template <typename T>
__device__ __forceinline__ float rest_of(float v) {
  const float r = v - (float)(T)v;
  return fabsf(r) < INFINITY ? r : 0.0f;
}

// LDS of a wave: each block of tokens, and a block of weights
constexpr int stream_bytes(int mt) { return (mt + 1) * kBlockBytes; }

template <class F, int MT, int NT, Tokens X = Tokens::Rows, typename T = void>
struct RowStream {
  static constexpr int XP = X == Tokens::Wide ? 2 : 1;  // 16-byte pieces of a token's share
  static constexpr int XL = X == Tokens::Wide ? 2 : 4;  // loads of a block of tokens, four of them each

  // Where the tokens and each block of weight rows start, the same for the wave,
  // and this lane's rows (4 i + l / 16 of each block) from there, below 2^31 bytes.
  const char *x, *w[NT];
  uint32_t xo[MT][XL], wo[NT][4];
  float scale[MT][XL];  // Wide: of x's rows
  // Rows of tokens there are.  The rows of a block past them are neither loaded nor put
  // into LDS: what they hold there reaches no token's sums.
  int have;

  int K, full;  // units of a row; whole blocks
  int piece;    // which 16 bytes of a row's block it loads
  char *put_at, *get_at;  // this lane's row in the wave's LDS, as it loads and as it multiplies
  int row, part;          // that row, and 16-byte piece
  f32x4 tot[MT][NT];
  u32x4 xr[MT][XL][XP], wr[NT][4];
  const char *xl;

  __device__ __forceinline__ void init(int lane, int units, char *lds) {
    K = units;
    full = units / 128;
    piece = lane & 15;
    put_at = lds + (lane >> 4) * 256;
    row = lane & 15;
    part = lane >> 4;
    get_at = lds + row * 256;
    clear();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int b = 0; b < NT; ++b) tot[m][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  __device__ __forceinline__ int blocks() const { return (K + 127) / 128; }

  // A lane's eight units of a row's block.  In the block that K ends in the
  // row's last eight, put in place when they are used.
  __device__ __forceinline__ int unit(int kb) const {
    const int k = kb * 128 + 8 * piece;
    return kb < full || k < K - 8 ? k : K - 8;
  }
  __device__ __forceinline__ u32x4 in_place(u32x4 v, int kb) const {
    if (kb >= full) {
      const int past = kb * 128 + 8 * piece - (K - 8);
      v = drop_values(v, past > 0 ? past : 0);
    }
    return v;
  }
  // Row 4 i + l / 16 of the wave's LDS: pieces in an order of the row's own, so
  // that the sixteen rows that a read touches lie on different banks.
  // Block `which` is the weights' at MT, else tokens'.
  __device__ __forceinline__ void put(int which, int i, u32x4 v) const {
    *reinterpret_cast<u32x4 *>(put_at + which * kBlockBytes + i * 1024 + ((piece ^ (4 * i + part)) * 16)) = v;
  }
  // A row of fp32 tokens' two.
  __device__ __forceinline__ void put_both(int which, int i, const u32x4 (&v)[2]) const {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      *reinterpret_cast<u32x4 *>(put_at + part * 256 + which * kBlockBytes + i * 2048 + r * 256 +
                                 ((piece ^ (8 * i + 2 * part + r)) * 16)) = v[r];
  }
  __device__ __forceinline__ u32x4 get(int which, int s) const {
    return *reinterpret_cast<const u32x4 *>(get_at + which * kBlockBytes + (((4 * s + part) ^ row) * 16));
  }

  __device__ __forceinline__ void load_x(int kb) {
    if constexpr (X == Tokens::Lds) return;
    const int k = unit(kb);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < XL; ++i) {
        if (4 * (XL * m + i) >= have) break;
        if constexpr (X == Tokens::Wide) {
          xr[m][i][0] = load_at<u32x4_any>(x, xo[m][i] + 4u * k);
          xr[m][i][1] = load_at<u32x4_any>(x, xo[m][i] + 4u * k + 16u);
        } else {
          xr[m][i][0] = load_at<u32x4_any>(x, xo[m][i] + 2u * k);
        }
      }
  }
  __device__ __forceinline__ void load_w(int b, int kb) {
    const int k = unit(kb);
#pragma unroll
    for (int i = 0; i < 4; ++i) wr[b][i] = load_at<u32x4_any>(w[b], wo[b][i] + 2u * k);
  }
  __device__ __forceinline__ void begin_weights(int kb) {
#pragma unroll
    for (int b = 0; b < NT; ++b) load_w(b, kb);
  }

  __device__ __forceinline__ void put_tokens(int m, int i, int kb) const {
    if constexpr (X == Tokens::Wide) {
      u32x4 v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f32x4 f = __builtin_bit_cast(f32x4, xr[m][i][e]);
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] *= scale[m][i];  // (times a vector of them, it is read from scratch memory)
        const u32x2 first = Mfma<T>::pack4(f[0], f[1], f[2], f[3]);
        const u32x2 rest = Mfma<T>::pack4(rest_of<T>(f[0]), rest_of<T>(f[1]), rest_of<T>(f[2]), rest_of<T>(f[3]));
        v[0][2 * e] = first[0];
        v[0][2 * e + 1] = first[1];
        v[1][2 * e] = rest[0];
        v[1][2 * e + 1] = rest[1];
      }
      v[0] = in_place(v[0], kb);
      v[1] = in_place(v[1], kb);
      put_both(m, i, v);
    } else {
      put(m, i, in_place(xr[m][i][0], kb));
    }
  }

  // All of rows shorter than eight units, value by value (not from LDS).
  __device__ __forceinline__ void short_rows() {
    u32x4 xs[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int i = 0; i < XL; ++i) {
        u32x4 v[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
        if constexpr (X == Tokens::Wide) {
          const float *from = reinterpret_cast<const float *>(x + xo[m][i]);
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (piece == 0 && e < K) {
              const float f = from[e] * scale[m][i];
              v[0][e / 2] |= Mfma<T>::pack4(f, 0.0f, 0.0f, 0.0f)[0] << (16 * (e % 2));
              v[1][e / 2] |= Mfma<T>::pack4(rest_of<T>(f), 0.0f, 0.0f, 0.0f)[0] << (16 * (e % 2));
            }
          put_both(0, i, v);
        } else {
          if (piece == 0) v[0] = load_tail(reinterpret_cast<const uint16_t *>(x + xo[m][i]), 0, K);
          put(0, i, v[0]);
        }
      }
      xs[m] = get(0, 0);
    }
#pragma unroll
    for (int b = 0; b < NT; ++b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (piece == 0) v = load_tail(reinterpret_cast<const uint16_t *>(w[b] + wo[b][i]), 0, K);
        put(MT, i, v);
      }
      const u32x4 ws = get(MT, 0);
#pragma unroll
      for (int m = 0; m < MT; ++m) tot[m][b] = F::mma(xs[m], ws, tot[m][b]);
    }
  }

  // Block kb, while block next loads (rows of eight units and more).
  template <bool MORE>
  __device__ __forceinline__ void block(int kb, int next) {
    if constexpr (X != Tokens::Lds) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < XL; ++i) {
          if (4 * (XL * m + i) >= have) break;
          put_tokens(m, i, kb);
        }
    }
    if (MORE) load_x(next);
#pragma unroll
    for (int b = 0; b < NT; ++b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) put(MT, i, in_place(wr[b][i], kb));
      if (MORE) load_w(b, next);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const u32x4 ws = get(MT, s);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const u32x4 xs = X == Tokens::Lds ? *reinterpret_cast<const u32x4 *>(xl + kb * 256 + s * 64) : get(m, s);
          tot[m][b] = F::mma(xs, ws, tot[m][b]);
        }
        if (s == 1) __builtin_amdgcn_sched_barrier(0);  // two steps' fragments at a time
      }
      __builtin_amdgcn_sched_barrier(0);
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
