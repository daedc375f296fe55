// A mixture-of-experts layer for few tokens:
//
//   l = x R^T, the top_k experts e of each token by l, p = softmax of l,
//   h_e = act(x Wg_e^T) * (x Wu_e^T),   y = sum over e of p_e h_e Wd_e^T.
//
// Bound by reading the reached experts' weights once.  Launches: the router's
// logits and the choice (together where the router is small), the gated blocks,
// the second products of each choice, and their sum (not for one choice).  Tokens
// are taken in chunks of 64, which do not know of each other.  A chunk has
// slots for the experts it may reach: one for each expert, or, where it has
// fewer choices than there are experts, one for each choice, used by the first
// choice of an expert.
#pragma once

#include "lane_ops.hpp"
#include "row_stream.hpp"
#include "serve.hpp"

namespace pgemm {

struct MoeArgs {
  const uint16_t *x, *router, *w, *down;
  uint16_t *y;
  int32_t *experts;    // [M][k]
  float *weights;      // [M][k]
  double *logits;      // [M][E]
  char *h;             // [M k][F] fp32 where T is f16, else [M k][2][F]: the values in T, and their rests
  uint32_t *tops;      // [M k] largest |h|, f16 only
  float *products;     // [M k][D] second products, times the choices' weights
  int M, E, D, F, k, slots;
  bool by_choice;      // slots are choices
  int act;
  bool normalize;
};

// The hidden values are multiplied again on the matrix units, as two numbers of
// 16 bits: what they round to in T, and what that leaves, rounded (2^-16 of them
// is lost in bf16, 2^-22 in f16; with the first alone results were off by half as
// much again as by their own rounding).  Both are rows of the second products,
// one after the other, and the sums of both are added at the end: eight tokens
// are a block of 16 rows.  One token's products take as long as with one part
// (16.5 us for 84 MB), since their rows were there.
// binary16 ends at 65504, which h may pass where y does not: in f16 they are
// kept in fp32 with each choice's largest, and split after a power of two that
// takes this into [2^14, 2^15).
template <typename T>
constexpr bool kWideHidden = std::is_same_v<T, _Float16>;

// ------------------------------------------------------------ the choice ---

// Logits in 64 bits, so that which experts a token gets depends on the order of
// the sum only where logits are some 2^-53 of their terms apart; equal router rows
// have equal logits.  A workgroup has one expert and up to TB tokens, a thread eight
// values of K at a time, two loads ahead.
template <typename T, int TB>
__global__ void __launch_bounds__(256) moe_logits_kernel(MoeArgs a) {
  __shared__ double sums[4][TB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x, m0 = blockIdx.y * TB;
  const uint16_t *r = a.router + (int64_t)e * a.D;
  double sum[TB];
#pragma unroll
  for (int i = 0; i < TB; ++i) sum[i] = 0.0;
  auto eight = [&](const uint16_t *row, int k) {
    if (k + 8 <= a.D) return (u32x4)*reinterpret_cast<const u32x4_any *>(row + k);
    return k < a.D ? load_tail(row, k, a.D) : u32x4{0u, 0u, 0u, 0u};
  };
  for (int k0 = 0; k0 < a.D; k0 += 4096) {
    u32x4 rv[2], xv[2][TB];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = k0 + j * 2048 + tid * 8;
      rv[j] = eight(r, k);
#pragma unroll
      for (int i = 0; i < TB; ++i) xv[j][i] = eight(a.x + (int64_t)(m0 + i < a.M ? m0 + i : a.M - 1) * a.D, k);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const double w = (double)widen<T>((uint16_t)(rv[j][n / 2] >> (16 * (n % 2))));
#pragma unroll
        for (int i = 0; i < TB; ++i)
          sum[i] = __builtin_fma((double)widen<T>((uint16_t)(xv[j][i][n / 2] >> (16 * (n % 2)))), w, sum[i]);
      }
  }
#pragma unroll
  for (int i = 0; i < TB; ++i) {
    sum[i] = wave_scan(sum[i]);
    if (lane == 63) sums[wave][i] = sum[i];
  }
  __syncthreads();
  if (tid < TB && m0 + tid < a.M)
    a.logits[(int64_t)(m0 + tid) * a.E + e] = (sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid]);
}

// Numbers as integers of the same order; a NaN is behind minus infinity.
__device__ __forceinline__ uint64_t moe_order(double v) {
  if (v != v) return 1;
  const uint64_t b = __builtin_bit_cast(uint64_t, v == 0.0 ? 0.0 : v);
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double moe_value(uint64_t o) {
  if (o == 1) return NAN;
  return __builtin_bit_cast(double, o >> 63 ? o ^ 1ull << 63 : ~o);
}

constexpr int kMoeChunk = kMoeChunkTokens;

// Top_k times the largest logit l that is left, the lowest index of equal ones, by
// one wave, for up to 64 PER experts; the sums' weights.
template <int PER>
__device__ __forceinline__ void moe_choose(const MoeArgs &a, const double *l, int m, int lane) {
  uint64_t left[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) left[i] = i * 64 + lane < a.E ? moe_order(l[i * 64 + lane]) : 0;
  double first = 0.0, mine = -INFINITY;
  int my_expert = 0;
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = left[0];
#pragma unroll
    for (int i = 1; i < PER; ++i)
      if (i * 64 < a.E && left[i] > best) best = left[i];
    best = wave_most(best);
    int at = -1;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * 64 < a.E && at < 0) {
        const uint64_t has = __ballot(left[i] == best);
        if (has) {
          at = i * 64 + __builtin_ctzll(has);
          if (lane == __builtin_ctzll(has)) left[i] = 0;
        }
      }
    const double v = moe_value(best);
    if (j == 0) first = v;
    if (lane == j) {
      mine = v;
      my_expert = at;
    }
  }
  mine = exp(mine - first);
  double total = 0.0;
  if (a.normalize)
    total = lane < a.k ? mine : 0.0;
  else
    for (int e = lane; e < a.E; e += 64) total += exp(l[e] - first);
  total = read_lane(wave_scan(total), 63);
  if (lane < a.k) {
    const int64_t at = (int64_t)m * a.k + lane;
    a.experts[at] = my_expert;
    a.weights[at] = (float)(mine / total);
    if (a.tops) a.tops[at] = 0;
  }
}

// A wave a token.
template <int PER>
__global__ void __launch_bounds__(64) moe_choose_kernel(MoeArgs a) {
  const int lane = threadIdx.x, m = blockIdx.x;
  moe_choose<PER>(a, a.logits + (int64_t)m * a.E, m, lane);
}

// Both for a token in one workgroup, where the router is small: its logits, an
// expert a wave, and then the choice.  One launch less: with 8 experts
// of 1024 values 3.5 us instead of 2.7 and 2.5.
constexpr int kMoeRouteExperts = 16, kMoeRouteValues = 4096;
template <typename T>
__global__ void __launch_bounds__(1024) moe_route_kernel(MoeArgs a) {
  __shared__ double logits[kMoeRouteExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = blockIdx.x;
  const uint16_t *x = a.x + (int64_t)m * a.D;
  auto eight = [&](const uint16_t *row, int k) {
    if (k + 8 <= a.D) return (u32x4)*reinterpret_cast<const u32x4_any *>(row + k);
    return k < a.D ? load_tail(row, k, a.D) : u32x4{0u, 0u, 0u, 0u};
  };
  for (int e = wave; e < a.E; e += 16) {
    const uint16_t *r = a.router + (int64_t)e * a.D;
    double sum = 0.0;
    for (int k0 = 0; k0 < a.D; k0 += 2048) {
      u32x4 xv[4], rv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * 512 + lane * 8;
        xv[j] = eight(x, k);
        rv[j] = eight(r, k);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int n = 0; n < 8; ++n)
          sum = __builtin_fma((double)widen<T>((uint16_t)(xv[j][n / 2] >> (16 * (n % 2)))),
                              (double)widen<T>((uint16_t)(rv[j][n / 2] >> (16 * (n % 2)))), sum);
    }
    sum = wave_scan(sum);
    if (lane == 63) logits[e] = sum;
  }
  __syncthreads();
  if (wave == 0) moe_choose<1>(a, logits, m, lane);
}

// ---------------------------------------------------------- the products ---

// The exponent of the factor of a choice's hidden values, from the largest one's bits.
__device__ __forceinline__ int moe_exponent(uint32_t top) {
  if (top == 0) return 0;
  int e;
  frexpf(__builtin_bit_cast(float, top), &e);
  return 15 - e > 127 ? 127 : 15 - e;
}

// waves a SIMD holds by their registers
constexpr int moe_per_simd(int mt) { return mt == 1 ? 4 : mt == 2 ? 3 : 2; }

// The gated blocks and, DOWN, the second products.  A workgroup has an expert's 16
// gate rows and the same 16 up rows, or 32 rows of its second matrix; its waves take blocks
// of K in turn and join their sums in LDS.  More than 16 MT tokens of an expert (DOWN:
// 8 MT) take another pass over these weights.  SHORT: rows of less than eight values.
//
// (Second products that a workgroup sums over all experts in LDS save the last
// launch, but leave little LDS for weights on the way, and few workgroups: 49 us
// instead of 46 and 5 for 37 tokens' four choices of 60 experts of 2048 x 1024 in
// bf16, 41 instead of 24 and 5 for 64 tokens' two of 8 of 4096 x 1280.)
//
// One token's eight choices of experts of 4096 x 1280: 31.5 us for 168 MB, 5.3 TB/s, and
// 16.5 us for 84 MB, 5.1 TB/s.  37 tokens' four of 60 of 2050 x 1001 in f16: 88 us for
// 450 MB, 5.1 TB/s, and 51 us for 225 MB, 4.4 TB/s, where weight rows start on odd
// multiples of two bytes and the tokens' are fp32.
template <typename T, int MT, int WAVES, bool DOWN, bool SHORT>
__global__ void __launch_bounds__(WAVES * 64, moe_per_simd(SHORT ? 4 : MT)) moe_rows_kernel(MoeArgs a) {
  constexpr int NT = 2, VALS = MT * NT * 4;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float *sums = reinterpret_cast<float *>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.y, chunk = blockIdx.z, n0 = blockIdx.x * (DOWN ? 32 : 16);
  const int t0 = chunk * kMoeChunk, tokens = a.M - t0 < kMoeChunk ? a.M - t0 : kMoeChunk;
  const int choices = tokens * a.k;
  const int32_t *experts = a.experts + (int64_t)t0 * a.k;
  if (a.by_choice && slot >= choices) return;  // a last chunk of few tokens
  const int expert = a.by_choice ? __builtin_amdgcn_readfirstlane(experts[slot]) : slot;
  const int K = DOWN ? a.F : a.D, rows = DOWN ? a.D : a.F;  // of a weight row; of a matrix
  constexpr bool WIDE = DOWN && kWideHidden<T>;
  constexpr int PARTS = DOWN ? 2 : 1;  // rows of a token
  using Stream = RowStream<Frag8<T>, MT, NT, WIDE ? Tokens::Wide : Tokens::Rows, T>;
  Stream job;
  char *mine = smem + wave * stream_bytes(MT);
  job.init(lane, K, mine);
  const int blocks = job.blocks(), turn = first_turn(blockIdx.x + slot * 7, blocks);
  auto block = [&](int i) { return i + turn < blocks ? i + turn : i + turn - blocks; };
  const uint16_t *w = DOWN ? a.down + (int64_t)expert * a.D * a.F : a.w + (int64_t)expert * 2 * a.F * a.D;
  const int64_t pitch = (int64_t)K * 2;
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    const int row0 = n0 + (DOWN ? 16 * b : 0);
    job.w[b] = block_start(w + (DOWN ? 0 : (int64_t)b * a.F * a.D), row0, rows, pitch);
#pragma unroll
    for (int i = 0; i < 4; ++i) job.wo[b][i] = block_row(row0, 4 * i + (lane >> 4), rows, pitch);
  }
  job.x = DOWN ? a.h + (int64_t)t0 * a.k * a.F * 4 : reinterpret_cast<const char *>(a.x + (int64_t)t0 * a.D);
  const bool streams = !SHORT && wave < blocks;
  // weights are on the way while the expert's tokens are found (a slot of a choice has some, but for a second choice of
  // its expert)
  if (a.by_choice && streams) job.begin_weights(block(wave));
  // The expert's choices, at most 64, one a lane, put in order by way of the wave's LDS.  (Kept in LDS beside the blocks
  // they took 144 bytes, for which a CU held one workgroup of four blocks of 16 rows instead of two: 64 tokens' two of 8
  // experts of 4096 x 1280 in bf16 86 us instead of 75.)
  uint16_t *list = reinterpret_cast<uint16_t *>(mine);
  int n = 0;
  bool taken = false;
  for (int base = 0; base < choices; base += 64) {
    const int c = base + lane;
    const bool is = c < choices && experts[c] == expert;
    const uint64_t who = __ballot(is);
    if (is) list[n + __popcll(who & ((1ull << lane) - 1))] = (uint16_t)c;
    if (a.by_choice) taken |= __ballot(is && c < slot) != 0;
    n += __popcll(who);
  }
  n = __builtin_amdgcn_readfirstlane(n);
  if (n == 0 || taken) return;
  const int listed = list[lane];
  auto choice_at = [&](int i) { return __shfl(listed, i < n ? i : n - 1); };

  const int c = lane & 15, q = lane >> 4;
  for (int first = 0; first < n; first += 16 * MT / PARTS) {
    job.have = (n - first) * (WIDE ? 1 : PARTS);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < Stream::XL; ++r) {
        const int row = 4 * (Stream::XL * m + r) + (lane >> 4), choice = choice_at(first + (WIDE ? row : row / PARTS));
        job.xo[m][r] = WIDE ? (uint32_t)choice * (uint32_t)K * 4u
                            : (uint32_t)(DOWN ? choice * PARTS + row % PARTS : choice / a.k) * (uint32_t)K * 2u;
        if constexpr (WIDE) job.scale[m][r] = ldexpf(1.0f, moe_exponent(a.tops[(int64_t)t0 * a.k + choice]));
      }
    job.clear();
    if constexpr (SHORT) {
      if (wave == 0 && K > 0) job.short_rows();
    } else if (streams) {
      int kb = block(wave);
      if (!a.by_choice || first > 0) job.begin_weights(kb);
      job.load_x(kb);
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
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) sums[(wave * VALS + (m * NT + b) * 4 + r) * 64 + lane] = job.tot[m][b][r];
    __syncthreads();
    constexpr int OB = DOWN ? NT : 1, TOKENS = 4 / PARTS;  // of a lane's four sums
    for (int i = wave; i < MT * OB * TOKENS; i += WAVES) {
      const int m = i / (OB * TOKENS), b = i / TOKENS % OB, r = i % TOKENS, col = n0 + 16 * b + c;
      const int place = first + (4 * m + q) * TOKENS + r;
      if (first + 4 * m * TOKENS + r >= n) continue;  // no token in any lane
      auto joined = [&](int of, int part) {
        float v = 0.0f;
#pragma unroll
        for (int u = 0; u < WAVES; ++u) v += sums[(u * VALS + (m * NT + of) * 4 + r * PARTS + part) * 64 + lane];
        return v;
      };
      const bool in = place < n && col < rows;
      const int64_t choice = (int64_t)t0 * a.k + choice_at(place);
      if constexpr (DOWN) {
        float v = joined(b, 0);
        const float rest = joined(b, 1);
        if (fabsf(v) < INFINITY) v += rest;  // an infinite weight's product has the value's sign, and not the rest's
        if constexpr (WIDE) v = ldexpf(v, -moe_exponent(a.tops[choice]));
        v *= a.weights[choice];
        if (in && a.k == 1)
          a.y[choice * a.D + col] = __builtin_bit_cast(uint16_t, (T)v);
        else if (in)
          a.products[choice * a.D + col] = v;
        continue;
      }
      const float h = activate(a.act, joined(0, 0)) * joined(1, 0);
      if constexpr (kWideHidden<T>) {
        if (in) reinterpret_cast<float *>(a.h)[choice * a.F + col] = h;
        // of the finite ones: the others end where the definition has them end
        uint32_t top = in && fabsf(h) < INFINITY ? __builtin_bit_cast(uint32_t, fabsf(h)) : 0u;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) {
          const uint32_t other = (uint32_t)__shfl_xor((int)top, d);
          top = other > top ? other : top;
        }
        if (c == 0 && place < n) atomicMax(a.tops + choice, top);
      } else {
        uint16_t *to = reinterpret_cast<uint16_t *>(a.h) + choice * 2 * a.F + col;
        if (in) {
          to[0] = __builtin_bit_cast(uint16_t, (T)h);
          to[a.F] = __builtin_bit_cast(uint16_t, (T)rest_of<T>(h));
        }
      }
    }
    __syncthreads();
  }
}

// y = the sum of a token's choices, in their order, four columns a thread.
template <typename T>
__global__ void __launch_bounds__(64) moe_sum_kernel(MoeArgs a) {
  typedef f32x4 __attribute__((aligned(4))) f32x4_any;
  const int per_row = (a.D + 3) / 4;
  const int64_t total = (int64_t)a.M * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 64) {
    const int64_t m = i / per_row;
    const int col = (int)(i % per_row) * 4;
    const float *from = a.products + m * a.k * a.D + col;
    uint16_t *to = a.y + m * a.D + col;
    if (col + 4 <= a.D) {
      f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int j0 = 0; j0 < a.k; j0 += 8) {  // eight loads on the way at once
        f32x4 p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          if (j0 + j < a.k) p[j] = *reinterpret_cast<const f32x4_any *>(from + (int64_t)(j0 + j) * a.D);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v += p[j];
      }
      *reinterpret_cast<u32x2_any *>(to) = Mfma<T>::pack4(v[0], v[1], v[2], v[3]);
    } else {
      for (int x = 0; col + x < a.D; ++x) {
        float v = 0.0f;
        for (int j = 0; j < a.k; ++j) v += from[(int64_t)j * a.D + x];
        to[x] = __builtin_bit_cast(uint16_t, (T)v);
      }
    }
  }
}

}  // namespace pgemm
