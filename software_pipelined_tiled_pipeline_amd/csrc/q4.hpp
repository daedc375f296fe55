// Products with few rows (tokens) and 4-bit weights with a scale and a zero
// point per group of a row: out = x W^T, or the gated block on such weights.
//
//   out[m][n] = sum over groups G of s[n][G] * sum over k in G of x[m][k] (q[n][k] - z[n][G])
//
// Bound by reading the weights once: two of them are a byte, so what a byte
// costs elsewhere counts four times as much as with 16-bit weights.  A lane
// that loads its own weight row's bytes makes every lane of a load a request of
// its own, about 50 a load: 24.6 us instead of 10 at 8192 x 8192.  So weights come
// in whole lines:
//
//  * weights: a wave's blocks of 32 weight rows and 128 k (2 KiB) go straight
//    into a ring of D slots in LDS, four lanes to a row's 64 bytes, and are
//    read from there as MFMA fragments, a dword of eight weights a lane;
//  * x: 16 lanes load a token's 128 k; they are put in the fragments' order
//    and written to LDS;
//  * scales and zero points of the workgroup's rows are kept in LDS, a dword
//    each, for CB blocks of K at a time.
//
// Waves: KW work on blocks of K in turn and join their sums in LDS at the end;
// NW beside each other on different weight rows share their tokens in LDS
// (worth it where more than 16 tokens would read the weights of many rows more
// than once).  MT blocks of 16 tokens; XI loads of four tokens each hold them.
//
// What is left is vector instructions.  Taking a block's 4096 weights apart is
// 72 (f16) or 56 (bf16) of them, a group's sums times its scale four for every
// 16 tokens and 16 weight rows; all of it is 170 to 380 for a block, beside 12
// to 40 MFMAs.  That is why what bf16 weights carry too much is taken off by
// MFMAs (48 x 4096 x 12288 gated, groups of 32, went from 43.6 us with a vector
// instruction for each accumulator to 37.5) and why scales are loaded four at a
// time (one at a time took 80 of 480 instructions).  Deeper rings (three and four
// slots for more than four tokens) changed nothing.  Measured with the weights
// of two calls in turn, which the last-level cache holds, and with those of so
// many that it does not: one token at 8192 x 8192 10.1 and 11.7 us (3.5 and 3.0
// TB/s); 48 x 4096 x 12288 gated in groups of 32 28.1 and 31.1 us in bf16, 25.2 in
// f16 with two.
#pragma once

#include "few_rows.hpp"

namespace pgemm {

struct Q4Args {
  const uint16_t *x;     // [M][K]
  const uint8_t *q;      // [rows][wb]
  const uint16_t *scale;  // [rows][groups]
  const uint8_t *zero;   // [rows][groups], or null (8 everywhere)
  uint16_t *out;         // [M][N]
  int M, N, K;           // N output columns; the gated block has 2 N weight rows
  int wb;                // bytes of a weight row
  int group, groups;
  uint64_t per32;        // u * per32 >> 40 is the group of k = 32 u (u up to 2^17)
  int sp;                // dwords of a row's scales in LDS, odd
  int act;
};

// waves a SIMD holds that LDS leaves room for
constexpr int q4_per_simd(int xi, int nw) { return nw == 3 ? 3 : nw > 1 ? 2 : xi == 1 ? 4 : 3; }

template <typename T, bool GATED, int MT, int GS, int XI, int NW, int KW, int D>
struct Q4Geom {
  static constexpr int NT = 2, WAVES = NW * KW, THREADS = WAVES * 64;
  static constexpr int ROWS = NW * 32;                  // weight rows of a workgroup
  static constexpr int COLS = GATED ? ROWS / 2 : ROWS;  // output columns
  static constexpr int CB = (NW == 1 ? 64 : NW < 4 ? 32 : 16) * GS;  // blocks of K whose scales are kept
  static constexpr int XBUFS = NW == 4 ? 2 : 1;
  static constexpr int RING = WAVES * D * 2048;
  static constexpr int XBYTES = KW * XBUFS * XI * 1024;
  static constexpr int XW = (XI + NW - 1) / NW;  // loads of x a wave does for a block
  static constexpr int JOIN = WAVES * MT * NT * 4 * 256;
  static_assert(D >= 2 && D <= 4, "");
  static_assert(CB % KW == 0 && (XI == 4 * MT || (MT == 1 && XI == 1)), "");
};

// One token's product with one weight row, as it is defined.  For rows shorter
// than eight values; and where weights that carry 16 + zero too much have summed
// up to what is not finite: an infinite x is then infinity less infinity, and
// values past 1e37 leave fp32 early.
template <typename T>
__device__ __forceinline__ float q4_dot(const Q4Args &a, int64_t m, int64_t row) {
  const uint16_t *x = a.x + m * a.K;
  const uint8_t *q = a.q + row * a.wb;
  float total = 0.0f, sum = 0.0f;
  for (int k0 = 0; k0 < a.K; k0 += 32) {
    const int g = (int)((uint64_t)(uint32_t)(k0 / 32) * a.per32 >> 40);
    const float z = a.zero ? (float)a.zero[row * a.groups + g] : 8.0f;
    if (k0 + 32 <= a.K) {
      // all in flight at once; eight bytes each: the kernels' tests count loads of sixteen
      u32x2 v[8], w[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = load_at<u32x2_any>(x, (uint32_t)(k0 + 4 * i) * 2u);
        compiler_fence();
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = load_at<u32x2>(q, (uint32_t)(k0 / 2 + 8 * i));
        compiler_fence();
      }
#pragma unroll
      for (int k = 0; k < 32; ++k)
        sum += widen<T>((uint16_t)(v[k / 4][k / 2 % 2] >> (16 * (k % 2)))) * ((float)(w[k / 16][k / 8 % 2] >> (k % 8 * 4) & 15u) - z);
    } else {
      for (int k = k0; k < a.K; ++k) sum += widen<T>(x[k]) * ((float)(q[k / 2] >> (4 * (k & 1)) & 15) - z);
    }
    if ((k0 + 32) % a.group == 0 || k0 + 32 >= a.K) {
      total += sum * widen<T>(a.scale[row * a.groups + g]);
      sum = 0.0f;
    }
  }
  return total;
}

template <typename T, bool GATED, int MT, int GS, int XI, int NW, int KW, int D>
__global__ void __launch_bounds__(NW *KW * 64, q4_per_simd(XI, NW)) q4_kernel(Q4Args a) {
  using G = Q4Geom<T, GATED, MT, GS, XI, NW, KW, D>;
  using F = Frag8<T>;
  constexpr int NT = G::NT, SG = 4 / GS, XW = G::XW, CB = G::CB;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave / NW, wn = wave % NW;
  const int c = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * G::COLS, m0 = blockIdx.y * MT * 16;

  char *ring = smem + wave * (D * 2048);
  char *xbuf = smem + G::RING + wk * (G::XBUFS * XI * 1024);
  uint32_t *scales = reinterpret_cast<uint32_t *>(smem + G::RING + G::XBYTES);

  // first matrix row and rows inside the matrix of this wave's block b
  auto block_row = [&](int w, int b, int *have) __attribute__((always_inline)) {
    const int n = n0 + (GATED ? w * 16 : w * 32 + b * 16);
    *have = a.N - n < 0 ? 0 : a.N - n < 16 ? a.N - n : 16;
    return (int64_t)n + (GATED && b ? a.N : 0);
  };

  // weights: lane l brings 16 bytes of row l / 4
  __amdgpu_buffer_rsrc_t rw[NT];
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    int have;
    const int64_t row = block_row(wn, b, &have);
    rw[b] = make_rsrc(wave_uniform(reinterpret_cast<const char *>(a.q) + (have ? row : 0) * a.wb),
                      (uint32_t)__builtin_amdgcn_readfirstlane(have * a.wb));
  }
  // the four 16-byte pieces of a row are kept in an order that spreads the
  // rows that a fragment read meets over the banks
  const uint32_t wvo = (uint32_t)(lane >> 2) * (uint32_t)a.wb + (uint32_t)(((lane & 3) ^ ((lane >> 4) & 3)) * 16);
  auto load_w = [&](int slot, int kb, bool there) __attribute__((always_inline)) {
    // bytes past the rows inside the matrix read zero, those past a row's end
    // (the next row's) meet x = 0
    const uint32_t off = there ? wvo + (uint32_t)kb * 64u : kOobOffset;
    load_lds_x4<0>(rw[0], ring + slot * 2048, off, 0);
    load_lds_x4<1>(rw[1], ring + slot * 2048, off, 0);
  };

  // x: lane l brings eight k of token l / 16 of each group of four
  const char *xrow[XW];
#pragma unroll
  for (int i = 0; i < XW; ++i) {
    const int m = m0 + 4 * (wn * XW + i) + (lane >> 4);
    xrow[i] = reinterpret_cast<const char *>(a.x + (int64_t)(m < a.M ? m : a.M - 1) * a.K);
  }
  const int blocks = (a.K + 127) / 128;
  // (K is at least eight: the row's last eight values are loaded where fewer
  // are left, and put in place when they are stored)
  auto load_x = [&](u32x4 (&to)[XW], int kb) __attribute__((always_inline)) {
    const int k = kb * 128 + 8 * (lane & 15);
    const uint32_t at = (uint32_t)(k < a.K - 8 ? k : a.K - 8) * 2u;
#pragma unroll
    for (int i = 0; i < XW; ++i) to[i] = load_at<u32x4_any>(xrow[i], at);
  };
  auto store_x = [&](char *to, u32x4 (&from)[XW], int kb) __attribute__((always_inline)) {
    if (kb * 128 + 128 > a.K) {
      const int k = kb * 128 + 8 * (lane & 15);
#pragma unroll
      for (int i = 0; i < XW; ++i) from[i] = drop_values(from[i], k > a.K - 8 ? k - (a.K - 8) : 0);
    }
#pragma unroll
    for (int i = 0; i < XW; ++i) {
      const int row = 4 * (wn * XW + i) + (lane >> 4);
      if (XI % NW != 0 && wn * XW + i >= XI) continue;
      *reinterpret_cast<u32x4 *>(to + row * 256 + (((lane & 15) ^ (row & 15)) * 16)) = weight_order(from[i]);
    }
  };

  f32x4 tot[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int b = 0; b < NT; ++b) tot[m][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const typename F::Bits bits;
  const uint32_t wread = c * 64 + q * 4;
  const int xr = XI < 4 ? c & (4 * XI - 1) : c;
  const uint32_t *myscales = scales + (wn * 32 + c) * a.sp;
  // Where the weights carry 16 + zero too much, the sums of x take it out
  // again: rows 4 g .. 4 g + 3 of `rows[g]` are ones, so that their products
  // with x leave the sum of x over group l / 16 of the block, token l % 16, in
  // lane l (zero past the last group): an operand of a product in fp32 with
  // scale (16 + zero).
  u32x4 rows[SG];
  if constexpr (!F::kExactZero) {
#pragma unroll
    for (int g = 0; g < SG; ++g) rows[g] = F::ones(c >> 2 == g);
  }

  auto compute = [&](const char *slot, const char *xs_, int kb, int g0) __attribute__((always_inline)) {
    uint32_t sv[SG][NT];
#pragma unroll
    for (int g = 0; g < SG; ++g) {
      const int gi = (int)((uint64_t)(uint32_t)(kb * 4 + GS * g) * a.per32 >> 40) - g0;
#pragma unroll
      for (int b = 0; b < NT; ++b) sv[g][b] = myscales[b * 16 * a.sp + gi];
    }
    f32x4 xs[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xs[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < SG; ++g) {
      f32x4 acc[MT][NT];
      typename F::Zero z[NT];
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        z[b].set(sv[g][b]);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int s = g * GS; s < (g + 1) * GS; ++s) {
        u32x4 xf[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          xf[m] = *reinterpret_cast<const u32x4 *>(xs_ + (16 * m + xr) * 256 + (((4 * s + q) ^ xr) * 16));
          if constexpr (!F::kExactZero) xs[m] = F::mma(rows[g], xf[m], xs[m]);
        }
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          const uint32_t v = *reinterpret_cast<const uint32_t *>(slot + b * 1024 + wread + ((s ^ (c >> 2)) * 16));
          const u32x4 f = F::weights(v, z[b], bits);
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[m][b] = F::mma(xf[m], f, acc[m][b]);
        }
      }
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const float sc = widen<T>((uint16_t)(sv[g][b] >> 16));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) tot[m][b][r] += sc * acc[m][b][r];
      }
    }
    if constexpr (!F::kExactZero) {
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        uint32_t v = sv[SG - 1][b];  // of group l / 16
#pragma unroll
        for (int g = 0; g < SG - 1; ++g) v = q == g ? sv[g][b] : v;
        const float off = F::excess(v);
#pragma unroll
        for (int m = 0; m < MT; ++m) tot[m][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(xs[m][0], off, tot[m][b], 0, 0, 0);
      }
    }
  };

  for (int c0 = 0; c0 < blocks; c0 += CB) {
    const int nb = blocks - c0 < CB ? blocks - c0 : CB;
    // Workgroups start at different blocks: rows are often a multiple of the
    // memory channels' interleave apart, and all would meet on the same few.
    const int turn = (int)((blockIdx.x * 0x9E3779B1u >> 12) % (unsigned)nb);
    const int mine = wk < nb ? (nb - wk + KW - 1) / KW : 0;
    const int rounds = NW == 1 ? mine : (nb + KW - 1) / KW;
    auto block = [&](int i) {
      const int p = mine > 0 ? wk + (i < mine ? i : mine - 1) * KW + turn : 0;
      return c0 + (p < nb ? p : p - nb);
    };
    // Loads are issued for every i, those past the last block with no bytes
    // (weights) or once more (x): the counts that the waits below rely on.
    u32x4 xreg[D - 1][XW];
#pragma unroll
    for (int i = 0; i < D - 1; ++i) {
      load_x(xreg[i], block(i));
      compiler_fence();
      load_w(i, block(i), i < mine);
      compiler_fence();
    }
    {
      const int g0 = (int)((uint64_t)(uint32_t)(c0 * 4) * a.per32 >> 40);
      const int ng = (int)((uint64_t)(uint32_t)((c0 + nb) * 4 - 1) * a.per32 >> 40) - g0 + 1;
      // KW * 2 threads a row, four groups each at a time.  Groups past the row's
      // end, whose products are zeros, get a scale of zero; rows past the
      // matrix, which reach no stored value, repeat its last one.
      constexpr int TPR = G::THREADS / G::ROWS;
      const int r = tid / TPR;
      int have;
      int64_t row = block_row(r / 32, r / 16 % 2, &have);
      row += have == 0 ? (int64_t)a.N - 1 - (row - (GATED && r / 16 % 2 ? a.N : 0)) : (r & 15) < have ? r & 15 : have - 1;
      const uint16_t *srow = a.scale + row * a.groups;
      const uint8_t *zrow = a.zero ? a.zero + row * a.groups : reinterpret_cast<const uint8_t *>(srow);
      uint32_t *to = scales + r * a.sp;
      auto stage = [&](int base, auto at_once) __attribute__((always_inline)) {
        constexpr int U = decltype(at_once)::value;
        uint64_t sv[U];
        uint32_t zv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int g = base + u * TPR * 4 + g0;
          if (a.groups >= 4) {
            const int at = g < a.groups - 4 ? g : a.groups - 4;
            sv[u] = load_at<u64_any>(srow, (uint32_t)at * 2u);
            zv[u] = load_at<u32_any>(zrow, (uint32_t)at);
          } else {  // one load has them all
            sv[u] = zv[u] = 0;
#pragma unroll
            for (int e = 0; e < 3; ++e) {
              const int at = e < a.groups ? e : a.groups - 1;
              sv[u] |= (uint64_t)(e < a.groups ? srow[at] : 0) << (16 * e);
              zv[u] |= (uint32_t)zrow[at] << (8 * e);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int g = base + u * TPR * 4;
          const int past = a.groups >= 4 ? g + g0 - (a.groups - 4) : g + g0;
          if (past > 0) {
            sv[u] = past < 4 ? sv[u] >> (16 * past) : 0;
            zv[u] = past < 4 ? zv[u] >> (8 * past) : 0;
          }
          if (g < ng) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              to[g + e] = F::pack((uint16_t)(sv[u] >> (16 * e)), a.zero ? zv[u] >> (8 * e) & 0xffu : 8u);
          }
        }
      };
      // several loads at once: one after the other would each wait for memory
      if (ng <= TPR * 4)
        stage(tid % TPR * 4, std::integral_constant<int, 1>{});
      else
        for (int base = tid % TPR * 4; base < ng; base += 4 * TPR * 4) stage(base, std::integral_constant<int, 4>{});
      // All loads so far are over: those of the last scales have come after them.
      // Said once more, because the compiler counts a load as in flight until a
      // wait on every path, and a thread with no scale to keep skips its own: it
      // then waited for all loads before each block's first MFMA.
      wait_vmcnt<0>();
      lds_barrier();
      // `behind`: how many blocks' loads follow this block's by the time it is
      // waited for.  The last D - 2 blocks load none of their own.
      auto round = [&](int i, u32x4(&x)[XW], auto behind) __attribute__((always_inline)) {
        constexpr int B = decltype(behind)::value;
        char *xs = xbuf + (G::XBUFS == 1 ? 0 : (i & 1)) * (XI * 1024);
        if (NW > 1 && G::XBUFS == 1) lds_barrier();  // the last block's tokens are no longer read
        store_x(xs, x, block(i));
        if constexpr (B == D - 1) {
          load_x(x, block(i + D - 1));
          wait_lgkmcnt0();  // the slot's last reads are over
          compiler_fence();
          load_w((i + D - 1) % D, block(i + D - 1), i + D - 1 < mine);
        }
        compiler_fence();
        wait_vmcnt<B *(XW + 2)>();
        compiler_fence();
        if (NW > 1) lds_barrier();
        if (NW == 1 || i < mine) compute(ring + (i % D) * 2048, xs, block(i), g0);
      };
      int i = 0;
      for (; i + D - 1 <= rounds; i += D - 1) {
#pragma unroll
        for (int j = 0; j < D - 1; ++j) round(i + j, xreg[j], std::integral_constant<int, D - 1>{});
      }
      if constexpr (D > 2)
        if (i < rounds) round(i, xreg[0], std::integral_constant<int, D - 2>{});
      if constexpr (D > 3)
        if (i + 1 < rounds) round(i + 1, xreg[1], std::integral_constant<int, D - 3>{});
    }
    wait_vmcnt<0>();
    // no load of x may be left out for being unused: the waits count them all
#pragma unroll
    for (int i = 0; i < D - 1; ++i)
#pragma unroll
      for (int k = 0; k < XW; ++k) asm volatile("" ::"v"(xreg[i][k]));
    __syncthreads();  // the ring, the tokens and the scales are free
  }

  float *sums = reinterpret_cast<float *>(smem) + wn * (MT * NT * 4 * 64);
  constexpr int PART = NW * MT * NT * 4 * 64;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[wk * PART + ((m * NT + b) * 4 + r) * 64 + lane] = tot[m][b][r];
  __syncthreads();
  join_and_store<T, GATED, MT, NT>(sums, KW, PART, wk, KW, lane, a.act, a.out, a.M, a.N, m0,
                                   n0 + wn * (GATED ? 16 : 32), [&](float v, int m, int64_t row) {
                                     if constexpr (F::kExactZero)
                                       return v;
                                     else
                                       return fabsf(v) < INFINITY ? v : q4_dot<T>(a, m, row);
                                   });
}

// Rows shorter than eight values: one output a thread.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256) q4_short_kernel(Q4Args a) {
  const int64_t total = (int64_t)a.M * a.N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / a.N, n = i % a.N;
    const float v = GATED ? activate(a.act, q4_dot<T>(a, m, n)) * q4_dot<T>(a, m, n + a.N) : q4_dot<T>(a, m, n);
    a.out[i] = __builtin_bit_cast(uint16_t, (T)v);
  }
}

}  // namespace pgemm
