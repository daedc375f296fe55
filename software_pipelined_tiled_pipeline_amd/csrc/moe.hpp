// A mixture-of-experts layer for few tokens:
//
//   l = x R^T, the top_k experts e of each token by l, p = softmax of l,
//   h_e = act(x Wg_e^T) * (x Wu_e^T),   y = sum over e of p_e h_e Wd_e^T.
//
// Bound by reading the reached experts' weights once.  Four launches: the
// router's logits, the choice, the gated blocks and the second products.  Tokens
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
  char *h;             // [M k][F]: T, or fp32 where T is f16
  uint32_t *tops;      // [M k] largest |h|, f16 only
  uint32_t *counts;    // [chunks][slots] choices of the slot's expert, and the expert << 8
  uint16_t *lists;     // [chunks][slots][64] which choices of the chunk they are
  float *partial;      // [splits][M][D] sums of y, if there are several
  uint32_t *arrived;   // [chunks][groups of 32 columns] workgroups of moe_down_kernel that are done
  int groups, splits;  // all of these groups; workgroups that share one
  int M, E, D, F, k, slots;
  bool by_choice;      // slots are choices
  int act;
  bool normalize;
};

// The hidden values are multiplied again on the matrix units and rounded to T
// for that.  binary16 ends at 65504, which h may pass where y does not: in f16
// they are kept in fp32 with each choice's largest, and rounded after a power
// of two that takes this into [2^14, 2^15).
template <typename T>
constexpr bool kWideHidden = std::is_same_v<T, _Float16>;

// ------------------------------------------------------------ the choice ---

// Logits in 64 bits: which experts a token gets must not depend on the order
// of the sum.  A workgroup has one expert and up to TB tokens, a thread eight
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

constexpr int kMoeChunk = kMoeChunkTokens, kMoeColumns = kMoeDownColumns;

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
  for (int i = m * 64 + lane; i < a.groups; i += a.M * 64) a.arrived[i] = 0;
  moe_choose<PER>(a, a.logits + (int64_t)m * a.E, m, lane);
}

// Both for a token in one workgroup, where the router is small: its logits, an
// expert a wave at a time, and then the choice.  One launch less: with 8 experts
// of 1024 values 3.5 us instead of 2.7 and 2.5.
constexpr int kMoeRouteExperts = 64, kMoeRouteValues = 65536;
template <typename T>
__global__ void __launch_bounds__(1024) moe_route_kernel(MoeArgs a) {
  __shared__ double logits[kMoeRouteExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = blockIdx.x;
  for (int i = m * 1024 + tid; i < a.groups; i += a.M * 1024) a.arrived[i] = 0;
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

// ---------------------------------------------------------- gated blocks ---

// A workgroup has an expert's 16 gate rows and the same 16 up rows; its waves
// take blocks of K in turn and join their sums in LDS.  More than 16 MT tokens
// of an expert take another pass over these weights.
// SHORT: D is below eight.
template <typename T, int MT, int WAVES, bool SHORT>
__global__ void __launch_bounds__(WAVES * 64, MT == 1 ? 4 : MT == 2 ? 3 : 2) moe_gated_kernel(MoeArgs a) {
  constexpr int NT = 2, VALS = MT * NT * 4;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  uint16_t *list = reinterpret_cast<uint16_t *>(smem);  // [64]
  int *found = reinterpret_cast<int *>(smem + 128);
  float *sums = reinterpret_cast<float *>(smem + 144);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.y, chunk = blockIdx.z, f0 = blockIdx.x * 16;
  const int t0 = chunk * kMoeChunk, tokens = a.M - t0 < kMoeChunk ? a.M - t0 : kMoeChunk;
  const int choices = tokens * a.k;
  const int32_t *experts = a.experts + (int64_t)t0 * a.k;
  if (a.by_choice && slot >= choices) {  // a last chunk of few tokens
    if (blockIdx.x == 0 && tid == 0) a.counts[(int64_t)chunk * a.slots + slot] = 0;
    return;
  }
  const int expert = a.by_choice ? __builtin_amdgcn_readfirstlane(experts[slot]) : slot;
  using Stream = RowStream<Frag8<T>, MT, NT>;
  Stream job;
  job.init(lane, a.D, reinterpret_cast<char *>(sums) + wave * stream_bytes(MT));
  const int blocks = job.blocks(), turn = first_turn(blockIdx.x + slot * 7, blocks);
  auto block = [&](int i) { return i + turn < blocks ? i + turn : i + turn - blocks; };
  const uint16_t *w = a.w + (int64_t)expert * 2 * a.F * a.D;
  const int64_t pitch = (int64_t)a.D * 2;
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    job.w[b] = block_start(w + (int64_t)b * a.F * a.D, f0, a.F, pitch);
#pragma unroll
    for (int i = 0; i < 4; ++i) job.wo[b][i] = block_row(f0, 4 * i + (lane >> 4), a.F, pitch);
  }
  job.x = reinterpret_cast<const char *>(a.x + (int64_t)t0 * a.D);
  const bool streams = !SHORT && wave < blocks;
  // weights are on the way while the expert's tokens are found (a slot of a choice has some, but for a second choice of
  // its expert)
  if (a.by_choice && streams) job.begin_weights(block(wave));
  if (wave == 0) {
    int n = 0;
    bool taken = false;  // an earlier choice has this expert's slot
    for (int base = 0; base < choices; base += 64) {
      const int c = base + lane;
      const bool is = c < choices && experts[c] == expert;
      const uint64_t who = __ballot(is);
      if (is) list[n + __popcll(who & ((1ull << lane) - 1))] = (uint16_t)c;
      if (a.by_choice) taken |= __ballot(is && c < slot) != 0;
      n += __popcll(who);
    }
    if (taken) n = 0;
    if (lane == 0) *found = n;
  }
  __syncthreads();
  const int n = __builtin_amdgcn_readfirstlane(*found);
  if (blockIdx.x == 0) {
    const int64_t at = (int64_t)chunk * a.slots + slot;
    if (tid == 0) a.counts[at] = (uint32_t)n | (uint32_t)expert << 8;
    if (tid < n) a.lists[at * kMoeChunk + tid] = list[tid];
  }
  if (n == 0) return;

  const int c = lane & 15, q = lane >> 4;
  auto same = []() {};
  for (int first = 0; first < n; first += 16 * MT) {
    job.have = n - first;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = first + 16 * m + 4 * r + (lane >> 4);
        job.xo[m][r] = (uint32_t)(list[i < n ? i : n - 1] / a.k * pitch);
      }
    job.clear();
    if constexpr (SHORT) {
      if (wave == 0 && a.D > 0) job.short_rows();
    } else if (streams) {
      int kb = block(wave);
      if (!a.by_choice || first > 0) job.begin_weights(kb);
      job.load_x(kb);
      for (int i = wave + WAVES; i < blocks; i += WAVES) {
        const int next = block(i);
        job.template block<true>(kb, next, same);
        kb = next;
      }
      job.template block<false>(kb, kb, same);
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) sums[(wave * VALS + (m * NT + b) * 4 + r) * 64 + lane] = job.tot[m][b][r];
    __syncthreads();
    for (int i = wave; i < MT * 4; i += WAVES) {
      const int m = i / 4, r = i % 4, place = first + 16 * m + 4 * q + r, col = f0 + c;
      if (first + 16 * m + r >= n) continue;  // no token in any lane
      auto joined = [&](int b) {
        float v = 0.0f;
#pragma unroll
        for (int u = 0; u < WAVES; ++u) v += sums[(u * VALS + (m * NT + b) * 4 + r) * 64 + lane];
        return v;
      };
      const float h = activate(a.act, joined(0)) * joined(1);
      const bool in = place < n && col < a.F;
      const int64_t choice = (int64_t)t0 * a.k + list[place < n ? place : n - 1];
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
        if (in) reinterpret_cast<uint16_t *>(a.h)[choice * a.F + col] = __builtin_bit_cast(uint16_t, (T)h);
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------- second products ---

// The exponent of the factor of a choice's hidden values, from the largest one's bits.
__device__ __forceinline__ int moe_exponent(uint32_t top) {
  if (top == 0) return 0;
  int e;
  frexpf(__builtin_bit_cast(float, top), &e);
  return 15 - e > 127 ? 127 : 15 - e;
}

__host__ __device__ constexpr int up_even(int n) { return (n + 1) & ~1; }
// LDS of moe_down_kernel
inline int moe_down_lds(int mt, int waves, int tokens, int k, int slots) {
  const int choices = tokens * k;
  return waves * (stream_bytes(mt) + tokens * kMoeColumns * 4) + choices * 12 + up_even(choices) * 2 + slots * 4 + 8 + choices;
}

// A workgroup has 32 columns of y and all experts of a chunk, or, with few
// columns, one of `splits` shares of them.  Their blocks of K, one expert's after
// the other's, are dealt to the waves in runs of the same length; where a run
// leaves an expert (or 16 MT of its tokens), the wave adds its sums, times the
// choices' weights, to its own copy of the chunk's rows.  The copies are added up
// in order at the end, and the shares by the workgroup that is done last.
// SHORT: F is below eight.
template <typename T, int MT, int WAVES, bool SHORT>
__global__ void __launch_bounds__(WAVES * 64, MT == 1 ? 4 : MT == 2 ? 3 : 2) moe_down_kernel(MoeArgs a) {
  constexpr int THREADS = WAVES * 64, AHEAD = 2, NT = kMoeColumns / 16;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int chunk = blockIdx.y, d0 = blockIdx.x * kMoeColumns, split = blockIdx.z;
  const int t0 = chunk * kMoeChunk, tokens = a.M - t0 < kMoeChunk ? a.M - t0 : kMoeChunk;
  const int choices = tokens * a.k;
  float *rows = reinterpret_cast<float *>(smem + WAVES * stream_bytes(MT));  // [WAVES][tokens][32]
  float *weight = rows + WAVES * tokens * kMoeColumns;                  // [choices]
  uint32_t *part = reinterpret_cast<uint32_t *>(weight + choices);      // [choices] of a part: first place in the list, how many << 16; expert
  uint16_t *list = reinterpret_cast<uint16_t *>(part + 2 * choices);    // [choices], by slot
  uint32_t *from_slot = reinterpret_cast<uint32_t *>(list + up_even(choices));  // [slots] first place in the list, how many << 16
  int *parts_found = reinterpret_cast<int *>(from_slot + a.slots), *last_one = parts_found + 1;
  int8_t *power = reinterpret_cast<int8_t *>(parts_found + 2);  // [choices] exponents (f16)

  // everything that is read here is on the way at once: the slots' lists before it is known how long they are
  const int blocks = (a.F + 127) / 128, quads = a.slots * (kMoeChunk / 4);  // four entries of the lists each
  const uint64_t *lists = reinterpret_cast<const uint64_t *>(a.lists + (int64_t)chunk * a.slots * kMoeChunk);
  uint64_t entries[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) entries[i] = tid + i * THREADS < quads && blocks > 0 ? lists[tid + i * THREADS] : 0;
  for (int i = tid; i < choices; i += THREADS) {
    const int64_t choice = (int64_t)t0 * a.k + i;
    weight[i] = a.weights[choice];
    if constexpr (kWideHidden<T>) power[i] = (int8_t)moe_exponent(blocks > 0 ? a.tops[choice] : 0);
  }
  for (int i = tid; i < WAVES * tokens * kMoeColumns; i += THREADS) rows[i] = 0.0f;
  if (wave == 0) {
    int at = 0, parts = 0;
    for (int base = 0; base < a.slots; base += 64) {
      const int s = base + lane;
      const uint32_t v = s < a.slots && blocks > 0 ? a.counts[(int64_t)chunk * a.slots + s] : 0u;
      const int n = (int)(v & 0xffu), mine = (n + 16 * MT - 1) / (16 * MT);
      const int before = (int)wave_scan((uint32_t)n), parts_before = (int)wave_scan((uint32_t)mine);
      const int to = at + before - n;
      if (s < a.slots) from_slot[s] = (uint32_t)to | (uint32_t)n << 16;
      for (int i = 0; i < mine; ++i) {
        const int left = n - i * 16 * MT;
        const int p = parts + parts_before - mine + i;
        part[2 * p] = (uint32_t)(to + i * 16 * MT) | (uint32_t)(left < 16 * MT ? left : 16 * MT) << 16;
        part[2 * p + 1] = v >> 8;
      }
      at += __builtin_amdgcn_readlane(before, 63);
      parts += __builtin_amdgcn_readlane(parts_before, 63);
    }
    if (lane == 0) *parts_found = parts;
  }
  __syncthreads();
  const int parts = __builtin_amdgcn_readfirstlane(*parts_found);
  for (int i = 0; i * THREADS < quads && parts > 0; ++i) {
    const int quad = tid + i * THREADS;
    if (quad >= quads) break;
    const uint32_t v = from_slot[quad / (kMoeChunk / 4)];
    const int first = quad % (kMoeChunk / 4) * 4, n = (int)(v >> 16);
    if (first >= n) continue;
    const uint64_t e = i == 0 ? entries[0] : i == 1 ? entries[1] : lists[quad];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (first + j < n) list[(v & 0xffffu) + first + j] = (uint16_t)(e >> (16 * j));
  }
  __syncthreads();

  using Stream = RowStream<Frag8<T>, MT, NT, kWideHidden<T> ? Tokens::Wide : Tokens::Rows, T>;
  Stream job;
  job.init(lane, a.F, smem + wave * stream_bytes(MT));
  const int64_t pitch = (int64_t)a.F * 2, total = (int64_t)parts * blocks;
  const int c = lane & 15, q = lane >> 4;
  const int share = split * WAVES + wave, shares = a.splits * WAVES;
  int64_t i = total * share / shares;
  const int64_t end = total * (share + 1) / shares;
  job.x = a.h + (int64_t)t0 * a.k * a.F * (kWideHidden<T> ? 4 : 2);
#pragma unroll
  for (int b = 0; b < NT; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) job.wo[b][r] = block_row(d0 + 16 * b, 4 * r + (lane >> 4), a.D, pitch);
  auto part_rows = [&](int g) __attribute__((always_inline)) {  // a part's rows
    const uint32_t v = part[2 * g];
    const int from = (int)(v & 0xffffu), n = __builtin_amdgcn_readfirstlane((int)(v >> 16));
    const int expert = __builtin_amdgcn_readfirstlane((int)part[2 * g + 1]);
    job.have = n;
    const uint16_t *down = a.down + (int64_t)expert * a.D * a.F;
#pragma unroll
    for (int b = 0; b < NT; ++b) job.w[b] = block_start(down, d0 + 16 * b, a.D, pitch);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * m + 4 * r + (lane >> 4), choice = list[from + (j < n ? j : n - 1)];
        job.xo[m][r] = (uint32_t)choice * (uint32_t)a.F * (kWideHidden<T> ? 4u : 2u);
        job.scale[m][r] = kWideHidden<T> ? ldexpf(1.0f, power[choice]) : 1.0f;
      }
  };
  auto add = [&](int g) __attribute__((always_inline)) {
    const uint32_t v = part[2 * g];
    const int from = (int)(v & 0xffffu), n = (int)(v >> 16);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * m + 4 * q + r;
        if (j >= n) continue;
        const int choice = list[from + j];
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          float s = job.tot[m][b][r];
          if constexpr (kWideHidden<T>) s = ldexpf(s, -power[choice]);
          rows[(wave * tokens + choice / a.k) * kMoeColumns + 16 * b + c] += weight[choice] * s;
        }
      }
    job.clear();
  };
  if constexpr (SHORT) {
    for (; i < end; ++i) {
      part_rows((int)i);
      job.short_rows();
      add((int)i);
    }
  } else if (i < end) {
    int g = __builtin_amdgcn_readfirstlane((int)(i / blocks)), kb = __builtin_amdgcn_readfirstlane((int)(i % blocks));
    auto same = []() {};
    part_rows(g);
    job.begin_weights(kb);
    job.load_x(kb);
    for (++i; i < end; ++i) {
      const bool leaves = kb + 1 == blocks;
      const int to = leaves ? 0 : kb + 1;
      job.template block<true>(kb, to, [&]() {
        if (leaves) part_rows(g + 1);
      });
      if (leaves) add(g++);
      kb = to;
    }
    job.template block<false>(kb, kb, same);
    add(g);
  }
  __syncthreads();
  for (int j = tid; j < tokens * kMoeColumns; j += THREADS) {
    const int col = d0 + j % kMoeColumns;
    if (col >= a.D) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += rows[w * tokens * kMoeColumns + j];
    const int64_t to = (int64_t)(t0 + j / kMoeColumns) * a.D + col;
    if (a.splits == 1)
      a.y[to] = __builtin_bit_cast(uint16_t, (T)v);
    else
      __hip_atomic_store(a.partial + (int64_t)split * a.M * a.D + to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (a.splits == 1) return;
  // The sums are stored and loaded by device-wide accesses, which no cache keeps to itself; each thread waits for its stores before the
  // workgroup arrives, and a share's loads come after all arrivals.  (Fences would write the whole of an L2 back: 150 us
  // instead of 20.)
  wait_vmcnt<0>();
  compiler_fence();
  __syncthreads();
  if (tid == 0)
    *last_one = __hip_atomic_fetch_add(a.arrived + chunk * gridDim.x + blockIdx.x, 1u, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)a.splits - 1;
  __syncthreads();
  if (!*last_one) return;
  compiler_fence();
  for (int j = tid; j < tokens * kMoeColumns; j += THREADS) {
    const int col = d0 + j % kMoeColumns;
    if (col >= a.D) continue;
    const int64_t to = (int64_t)(t0 + j / kMoeColumns) * a.D + col;
    float v = 0.0f;
    for (int i = 0; i < a.splits; ++i)
      v += __hip_atomic_load(a.partial + (int64_t)i * a.M * a.D + to, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    a.y[to] = __builtin_bit_cast(uint16_t, (T)v);
  }
}

}  // namespace pgemm
