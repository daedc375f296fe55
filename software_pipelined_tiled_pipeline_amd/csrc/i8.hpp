// Products of 8-bit integers with a scale for each token and each weight row:
//
//   out[m][n] = xs[m] ws[n] * sum over k of x[m][k] w[n][k]
//
// and the gated block on them.  Sums are int32 and exact (widths end where
// 128 * 128 * K could leave it); the scales are applied in fp32 once.
// Rows are padded to 16 bytes, with zeros on the tokens' side.
#pragma once

#include "fused_launch.hpp"
#include "row_stream.hpp"

namespace pgemm {

// The integers' row width in bytes.
inline int64_t i8_width(int64_t K) { return up_to(K, 16); }

// acc xs ws without leaving fp32 where the result does not: a scale of at most
// 1 comes first, after which the sum is below 2^31; above 1 it comes last,
// where it overflows only if the result does.  What falls below 2^-126 on the
// way is an integer times a subnormal scale, and exact.
__device__ __forceinline__ float i8_scaled(int acc, float xs, float ws) {
  const float a = (float)acc;
  const bool small = fabsf(xs) <= 1.0f;
  return a * (small ? xs : ws) * (small ? ws : xs);
}

// --------------------------------------------------------- quantization ---

// A row's scale from its largest magnitude, at least the smallest normal
// number; NaN for a row that holds an infinity or a NaN.
__device__ __forceinline__ float i8_scale(float top) {
  return top < INFINITY ? fmaxf(top / 127.0f, 0x1p-126f) : NAN;
}

// Whether a row holds an infinity or a NaN shows in the largest of its
// magnitudes' bits, which have their values' order: two at a time.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
struct Largest {
  u16x2 top = {0, 0};
  __device__ __forceinline__ void take(const u32x4 &v) {
#pragma unroll
    for (int d = 0; d < 4; ++d) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, v[d] & 0x7FFF7FFFu));
  }
  __device__ __forceinline__ uint32_t bits() const { return top[0] > top[1] ? top[0] : top[1]; }
};
template <typename T>
__device__ __forceinline__ float i8_scale_of(uint32_t bits) {
  return i8_scale(bits < (std::is_same_v<T, _Float16> ? 0x7C00u : 0x7F80u) ? widen<T>((uint16_t)bits) : INFINITY);
}
__device__ __forceinline__ uint32_t wave_largest(uint32_t top) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, d);
    top = o > top ? o : top;
  }
  return top;
}

// x / s rounded to the nearest integer n, to the even one of two, by the sign
// of what x is above n s or below it and half an s more: exact, since x has at
// most 11 bits, n s at most 31, and their difference is about s / 2.
__device__ __forceinline__ int i8_quantized(float x, float s, float inverse) {
  const float n = __builtin_rintf(x * inverse);
  const float twice = 2.0f * __builtin_fmaf(-n, s, x);
  const bool odd = ((int)n & 1) != 0;
  float to = n;
  if (twice > s || (twice == s && odd)) to += 1.0f;
  if (twice < -s || (twice == -s && odd)) to -= 1.0f;
  return (int)to;
}

// Eight values' integers.  x times the reciprocal is within 2^-16 of the
// quotient (|x / s| <= 127, two roundings of 2^-24), so that its nearest integer is the
// right one unless it lies that near to a half, where i8_quantized takes over.
// 1.5 * 2^23 added to it leaves the integer in the lowest byte.  Beyond 127 it
// does not come: s is at least (1 - 2^-24) max |x| / 127.
template <typename T>
__device__ __forceinline__ u32x2 i8_packed(const u32x4 &v, float s, float inverse) {
  constexpr float MAGIC = 12582912.0f, NEAR = 0.5f - 0x1p-15f;
  uint32_t q[8];
  float off = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = widen<T>((uint16_t)(v[e / 2] >> (16 * (e % 2))));
    const float f = __builtin_fmaf(x, inverse, MAGIC);
    q[e] = __builtin_bit_cast(uint32_t, f);
    off = fmaxf(off, fabsf(__builtin_fmaf(x, inverse, MAGIC - f)));
  }
  if (!(off < NEAR)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = (uint32_t)i8_quantized(widen<T>((uint16_t)(v[e / 2] >> (16 * (e % 2)))), s, inverse);
  }
  u32x2 p;
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    const uint32_t lo = __builtin_amdgcn_perm(q[e + 1], q[e], 0x0c0c0400u), hi = __builtin_amdgcn_perm(q[e + 3], q[e + 2], 0x04000c0cu);
    p[e / 4] = lo | hi;
  }
  return s == s ? p : u32x2{0u, 0u};
}

// Eight values of a row from k on, zeros from K on (K at least eight).
__device__ __forceinline__ u32x4 load_eight(const uint16_t *row, int k, int K) {
  if (k >= K) return u32x4{0u, 0u, 0u, 0u};
  const int at = k < K - 8 ? k : K - 8;
  const u32x4 v = *reinterpret_cast<const u32x4_any *>(row + at);
  return k > at ? drop_values(v, k - at) : v;
}

// Rows shorter than eight values, one a thread.
template <typename T>
__global__ void __launch_bounds__(256) quant_short_kernel(const uint16_t *__restrict__ x, int8_t *__restrict__ q,
                                                          float *__restrict__ scale, int64_t M, int K) {
  for (int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x; m < M; m += (int64_t)gridDim.x * 256) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (K > 0) v = load_tail(x + m * K, 0, K);
    Largest top;
    top.take(v);
    const float s = i8_scale_of<T>(top.bits());
    const u32x2 p = i8_packed<T>(v, s, 1.0f / s);
    scale[m] = s;
    if (K > 0) *reinterpret_cast<u32x4 *>(q + m * 16) = u32x4{p[0], p[1], 0u, 0u};
  }
}

// WAVES waves a row, which is kept in registers between its maximum and its
// integers where it has up to 512 WAVES C values; longer rows are read twice.
// Bound by memory: 12288 x 4096 in bf16 24 us (6.2 TB/s read and written), 8192 x 8192
// 40 us.  With the exact division's correction for every value (i8_quantized)
// it was bound by vector instructions: 61 and 167 us.
template <typename T, int WAVES, int C>
__global__ void __launch_bounds__(256, 6) quant_rows_kernel(const uint16_t *__restrict__ x, int8_t *__restrict__ q,
                                                            float *__restrict__ scale, int64_t M, int K, int width) {
  constexpr int THREADS = WAVES * 64, ROWS = 4 / WAVES;  // of a workgroup
  __shared__ uint32_t tops[2][4];
  const int tid = threadIdx.x % THREADS, wave = threadIdx.x >> 6;
  int turn = 0;
  for (int64_t m0 = (int64_t)blockIdx.x * ROWS; m0 < M; m0 += (int64_t)gridDim.x * ROWS, turn ^= 1) {
    const int64_t m = m0 + threadIdx.x / THREADS;
    if (WAVES == 1 && m >= M) continue;
    const uint16_t *row = x + m * K;
    int8_t *to = q + m * width;
    u32x4 v[C];
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = load_eight(row, (i * THREADS + tid) * 8, K);
    Largest top;
#pragma unroll
    for (int i = 0; i < C; ++i) top.take(v[i]);
    for (int k = (C * THREADS + tid) * 8; k < K; k += THREADS * 8) top.take(load_eight(row, k, K));
    uint32_t bits = wave_largest(top.bits());
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) tops[turn][wave] = bits;
      __syncthreads();  // one a turn: the next one's values go to the other half
#pragma unroll
      for (int w = 0; w < WAVES; ++w) bits = tops[turn][w] > bits ? tops[turn][w] : bits;
    }
    const float s = i8_scale_of<T>(bits), inverse = 1.0f / s;
    if (tid == 0) scale[m] = s;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int k = (i * THREADS + tid) * 8;
      if (k < width) *reinterpret_cast<u32x2 *>(to + k) = i8_packed<T>(v[i], s, inverse);
    }
    for (int k = (C * THREADS + tid) * 8; k < width; k += THREADS * 8)
      *reinterpret_cast<u32x2 *>(to + k) = i8_packed<T>(load_eight(row, k, K), s, inverse);
  }
}

// ------------------------------------------------------------ few tokens ---

struct I8Args {
  const uint16_t *x;  // [M][K], or null:
  const int8_t *q;    // [M][width]
  const float *xs;    // [M]
  const int8_t *w;    // [N or 2 N][width]
  const float *ws;
  uint16_t *out;  // [M][N]
  int M, N, K, width;
  int act;
};

constexpr int kI8OwnTokens = 4;     // tokens that a workgroup makes integers of itself,
constexpr int kI8OwnWidth = 8192;   // of at most so many values

// LDS of a workgroup's sums, and of its waves' blocks before
constexpr int i8_sums(int mt, int waves, bool own) {
  return waves * (mt * 2048 > stream_bytes(own ? 0 : mt) ? mt * 2048 : stream_bytes(own ? 0 : mt));
}

// A workgroup has 32 weight rows (16 of the gate and the same 16 of the up
// projection) and all of K; its waves take blocks of 256 bytes in turn and add
// their sums up in LDS.  XL: tokens of 16 bits are made integers by every
// workgroup for itself while its first weights are on the way, which saves a
// launch (about 4 us).
// Bound by reading the weights: one token, gated, 12288 x 4096 in bf16 16.7 us for 101 MB
// (6.0 TB/s), 13 tokens at 11001 x 4090 in f16 10.0 us for 45 MB; with each lane on a row
// of its own, 64 bytes at a time, 18.2 and 11.0.  Eight waves along K up to 512
// workgroups, so that two a CU have 16 waves between them; four above, where the CUs
// have as many from more workgroups and fewer sums are joined.
template <typename T, bool GATED, int MT, int WAVES, bool XL>
__global__ void __launch_bounds__(WAVES * 64) i8_few_kernel(I8Args a) {
  constexpr int NT = 2, THREADS = WAVES * 64, VALS = MT * NT * 4;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * (GATED ? 16 : 32), m0 = blockIdx.y * MT * 16;
  float *scales = reinterpret_cast<float *>(smem);  // XL: the tokens' scales
  int *sums = reinterpret_cast<int *>(smem + (XL ? 64 : 0));
  constexpr int STREAM = stream_bytes(XL ? 0 : MT), SUMS = i8_sums(MT, WAVES, XL);  // and the waves' blocks before
  char *tokens = smem + 64 + SUMS;

  using Stream = RowStream<Int8Step, MT, NT, XL ? Tokens::Lds : Tokens::Rows>;
  Stream job;
  job.init(lane, a.width / 2, reinterpret_cast<char *>(sums) + wave * STREAM - (XL ? MT * kBlockBytes : 0));
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    const int row0 = n0 + (GATED ? 0 : 16 * b);
    job.w[b] = block_start(a.w + (GATED && b ? (int64_t)a.N * a.width : 0), row0, a.N, a.width);
#pragma unroll
    for (int i = 0; i < 4; ++i) job.wo[b][i] = block_row(row0, 4 * i + (lane >> 4), a.N, a.width);
  }
  job.have = a.M - m0;
  job.x = XL ? nullptr : block_start(a.q, m0, a.M, a.width);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) job.xo[m][i] = block_row(m0, 16 * m + 4 * i + (lane >> 4), a.M, a.width);
  const int blocks = job.blocks(), turn = first_turn(blockIdx.x, blocks);
  auto block = [&](int i) { return i + turn < blocks ? i + turn : i + turn - blocks; };
  int kb = wave < blocks ? block(wave) : 0;

  if constexpr (XL) {
    constexpr int C = kI8OwnWidth / (THREADS * 8);
    static_assert(C * THREADS * 8 == kI8OwnWidth && kI8OwnTokens * 4 <= kBlockBytes, "");
    const int pitch = blocks * 256 + 16;
    u32x4 v[kI8OwnTokens][C];
#pragma unroll
    for (int m = 0; m < kI8OwnTokens; ++m)
#pragma unroll
      for (int i = 0; i < C; ++i)
        v[m][i] = m < a.M ? load_eight(a.x + (int64_t)m * a.K, (i * THREADS + tid) * 8, a.K) : u32x4{0u, 0u, 0u, 0u};
    compiler_fence();  // the tokens first: waiting for them is then not waiting for the weights
    if (wave < blocks) job.begin_weights(kb);
    compiler_fence();
    uint32_t *tops = reinterpret_cast<uint32_t *>(sums);  // [tokens][waves]
#pragma unroll
    for (int m = 0; m < kI8OwnTokens; ++m) {
      if (m >= a.M) continue;
      Largest top;
#pragma unroll
      for (int i = 0; i < C; ++i) top.take(v[m][i]);
      const uint32_t bits = wave_largest(top.bits());
      if (lane == 0) tops[m * WAVES + wave] = bits;
    }
    lds_barrier();
#pragma unroll
    for (int m = 0; m < kI8OwnTokens; ++m) {
      if (m >= a.M) continue;
      uint32_t bits = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) bits = tops[m * WAVES + w] > bits ? tops[m * WAVES + w] : bits;
      const float s = i8_scale_of<T>(bits), inverse = 1.0f / s;
      if (tid == 0) scales[m] = s;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int k = (i * THREADS + tid) * 8;
        if (k < blocks * 256) *reinterpret_cast<u32x2 *>(tokens + m * pitch + k) = i8_packed<T>(v[m][i], s, inverse);
      }
    }
    lds_barrier();
    const int row = lane & 15;
    job.xl = tokens + (row < a.M ? row : a.M - 1) * pitch + 16 * (lane >> 4);
  } else {
    if (wave < blocks) {
      job.begin_weights(kb);
      job.load_x(kb);
    }
  }
  if (wave < blocks) {
    for (int i = wave + WAVES; i < blocks; i += WAVES) {
      const int next = block(i);
      job.template block<true>(kb, next);
      kb = next;
    }
    job.template block<false>(kb, kb);
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int b = 0; b < NT; ++b) {
      const i32x4 v = __builtin_bit_cast(i32x4, job.tot[m][b]);
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[(wave * VALS + (m * NT + b) * 4 + r) * 64 + lane] = v[r];
    }
  __syncthreads();

  constexpr int OB = GATED ? 1 : NT;
  const int c = lane & 15, q = lane >> 4;
  for (int i = wave; i < MT * OB * 4; i += WAVES) {
    const int m = i / (OB * 4), b = i / 4 % OB, r = i % 4;
    const int row = m0 + 16 * m + 4 * q + r, col = n0 + 16 * b + c;
    if (row >= a.M || col >= a.N) continue;
    auto joined = [&](int block) {
      int v = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v += sums[(w * VALS + (m * NT + block) * 4 + r) * 64 + lane];
      return v;
    };
    const float xs = XL ? scales[row] : a.xs[row];
    float v = i8_scaled(joined(b), xs, a.ws[col]);
    if constexpr (GATED) v = activate(a.act, v) * i8_scaled(joined(1), xs, a.ws[(int64_t)col + a.N]);
    a.out[(int64_t)row * a.N + col] = __builtin_bit_cast(uint16_t, (T)v);
  }
}

// ------------------------------------------------------------ many tokens ---
//
// The tiled product (fused_gemm.hpp) on rows of bytes: a granule of 16 bytes
// holds 16 integers of K instead of eight values, and
// v_mfma_i32_16x16x64_i8 takes as long as v_mfma_f32_16x16x32 with twice the
// operations.  Accumulators keep int32 bits.  Bound by the matrix units and the
// board's power: 8192 x 8192 x 8192 400 us (2.75 POP/s), 2048 x 4096 x 8192 gated
// 112 us (2.45 POP/s).

template <>
struct Mfma<int8_t> {
  template <bool ACC_AGPR>
  __device__ __forceinline__ static void run(u32x4 src0, u32x4 src1, f32x4 &acc) {
    if constexpr (ACC_AGPR)
      asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(src0), "v"(src1));
    else
      asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+v"(acc) : "v"(src0), "v"(src1));
  }
};

// A lane's column scales, those past the matrix's last column repeated.
__device__ __forceinline__ f32x4 i8_column_scales(const float *ws, int col, int N) {
  f32x4 v;
#pragma unroll
  for (int x = 0; x < 4; ++x) v[x] = ws[col + x < N ? col + x : N - 1];
  return v;
}

template <typename O>
struct I8Epi {
  struct Args {
    uint16_t *out;
    const float *xs, *ws;
  };
  template <typename T, class G, class W>
  struct Run {
    __device__ __forceinline__ void operator()(W &w, const Args &e, const FusedProduct &g, char *smem, int m0, int n0,
                                               int wm, int wn, int lane, int tid) const {
      constexpr int PITCH = Staging<G::BN>::PITCH;
      const int lr = wm * G::WM + (lane & 15), lc = wn * G::WN + 4 * (lane >> 4);
      float xs[W::TM];
#pragma unroll
      for (int i = 0; i < W::TM; ++i) xs[i] = e.xs[m0 + lr + 16 * i < g.M ? m0 + lr + 16 * i : g.M - 1];
#pragma unroll
      for (int j = 0; j < W::TN; ++j) {
        const f32x4 ws = i8_column_scales(e.ws, n0 + lc + 16 * j, g.N);
#pragma unroll
        for (int i = 0; i < W::TM; ++i) {
          const i32x4 v = __builtin_bit_cast(i32x4, w.acc[i][j]);
          *reinterpret_cast<u32x2 *>(smem + (lr + 16 * i) * PITCH + (lc + 16 * j) * 2) =
              Mfma<O>::pack4(i8_scaled(v[0], xs[i], ws[0]), i8_scaled(v[1], xs[i], ws[1]), i8_scaled(v[2], xs[i], ws[2]),
                             i8_scaled(v[3], xs[i], ws[3]));
        }
      }
      __syncthreads();
      store_tile<G::BM, G::BN, G::THREADS>(smem, PITCH, 0, e.out, g.N, g.M, g.N, m0, n0, tid);
    }
  };
};

template <typename O>
struct I8GatedEpi {
  struct Args {
    uint16_t *out;
    const float *xs, *ws;
    int act;
  };
  template <typename T, class G, class W>
  struct Run {
    __device__ __forceinline__ void operator()(W &w, const Args &e, const FusedProduct &g, char *smem, int m0, int n0,
                                               int wm, int wn, int lane, int tid) const {
      constexpr int ON = G::BN / 2, PITCH = Staging<ON>::PITCH;
      const int r = lane & 15, q = lane >> 4;
      float xs[W::TM];
#pragma unroll
      for (int i = 0; i < W::TM; ++i) {
        const int row = m0 + wm * G::WM + 16 * i + r;
        xs[i] = e.xs[row < g.M ? row : g.M - 1];
      }
#pragma unroll
      for (int p = 0; p < W::TN / 2; ++p) {
        const int lcol = wn * (G::WN / 2) + 16 * p + 4 * q;
        const f32x4 wg = i8_column_scales(e.ws, n0 + lcol, g.N), wu = i8_column_scales(e.ws + g.N, n0 + lcol, g.N);
#pragma unroll
        for (int i = 0; i < W::TM; ++i) {
          const i32x4 ga = __builtin_bit_cast(i32x4, w.acc[i][2 * p]), up = __builtin_bit_cast(i32x4, w.acc[i][2 * p + 1]);
          f32x4 h;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            h[x] = activate(e.act, i8_scaled(ga[x], xs[i], wg[x])) * i8_scaled(up[x], xs[i], wu[x]);
          *reinterpret_cast<u32x2 *>(smem + (wm * G::WM + 16 * i + r) * PITCH + lcol * 2) = Mfma<O>::pack4(h[0], h[1], h[2], h[3]);
        }
      }
      __syncthreads();
      store_tile<G::BM, ON, G::THREADS>(smem, PITCH, 0, e.out, g.N, g.M, g.N, m0, n0, tid);
    }
  };
};

// A piece of K: the sums as they are, for i8_join_kernel.
struct I8PieceEpi {
  struct Args {
    int *part;  // [pieces][M][pp]
    int pp;     // a multiple of 4
  };
  template <typename T, class G, class W>
  struct Run {
    __device__ __forceinline__ void operator()(W &w, const Args &e, const FusedProduct &g, char *smem, int m0, int n0,
                                               int wm, int wn, int lane, int tid) const {
      int *part = e.part + (int64_t)g.piece * g.M * e.pp;
#pragma unroll
      for (int i = 0; i < W::TM; ++i) {
        const int row = m0 + wm * G::WM + 16 * i + (lane & 15);
        if (row >= g.M) continue;
#pragma unroll
        for (int j = 0; j < W::TN; ++j) {
          const int col = n0 + wn * G::WN + 16 * j + 4 * (lane >> 4);
          if (col < g.N) *reinterpret_cast<f32x4 *>(part + (int64_t)row * e.pp + col) = w.acc[i][j];
        }
      }
    }
  };
};

template <typename O>
__global__ void __launch_bounds__(256) i8_join_kernel(const int *__restrict__ part, int pieces, int M, int N, int pp,
                                                      const float *__restrict__ xs, const float *__restrict__ ws,
                                                      uint16_t *__restrict__ out) {
  const int per_row = pp / 4;
  const int64_t total = (int64_t)M * per_row, stride = (int64_t)M * pp;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_row;
    const int col = (int)(i % per_row) * 4;
    i32x4 v = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < pieces; ++s) v += *reinterpret_cast<const i32x4 *>(part + i * 4 + s * stride);
    const f32x4 w = i8_column_scales(ws, col, N);
    const float x = xs[row];
    const u32x2 r = Mfma<O>::pack4(i8_scaled(v[0], x, w[0]), i8_scaled(v[1], x, w[1]), i8_scaled(v[2], x, w[2]),
                                   i8_scaled(v[3], x, w[3]));
    uint16_t *dst = out + row * N + col;
    if (col + 4 <= N) {
      *reinterpret_cast<u32x2_any *>(dst) = r;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < N) dst[e] = (uint16_t)(r[e / 2] >> (16 * (e % 2)));
    }
  }
}

}  // namespace pgemm
