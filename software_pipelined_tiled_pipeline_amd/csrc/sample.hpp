// One token for each row of logits, from a given random number.
//
// The tokens of a row in order: the largest logit first, the lowest index of
// equal ones.  With e_i = e^((z_i - z_1) / temperature) and S_n the sum of the
// first n of them, what is kept is the first
//   n = min(top_k, the fewest with S_n >= top_p S_top_k, how many have e_i >= min_p),
// at least one, and the token is the first of these with S_i > u S_n.
//
// Logits of 16 bits have few values, so that every such sum is one over values
// and not over tokens: a row is counted by value, and a value's share is its
// count times one exponential.  Counts do not depend on the order of their
// atomics, and all sums are in 64 bits.
//
// A workgroup has a row.  (Several could count one, since the blocks' counts and
// sums of shares below are linear in the counts, and would join 12 KiB each; values
// are needed one by one only where a border falls.)
// Bound by a CU's own time: of 24 us for one row of 131072 logits in bf16 about 9
// for reading and counting (vector instructions, two logits a dozen), 5 for the
// blocks' sums and shares, 5 for one wave's search for the borders of what is
// kept, 3 for finding the token's index; 256 rows of 50021 in f16, one a CU, 23 us.
// (First reading a row for its maximum, then counting below it, with an
// exponential a value, took 121 and 157 us.)
#pragma once

#include "fused_launch.hpp"
#include "lane_ops.hpp"
#include "serve.hpp"

namespace pgemm {

struct SampleArgs {
  const uint16_t *logits;  // [M][V]
  const float *u, *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p;
  int64_t *token;
  int64_t M;
  int V;
  int shared;  // bits: one value for all rows
};

constexpr int kSampleThreads = 1024, kSampleWaves = kSampleThreads / 64;
// LDS holds the counts of all values there are, two of 16 bits in a dword: 64
// values whose bits follow each other share 32 dwords, which are in an order of
// their block's own, so that a wave's reads fall on different banks.  The
// place is made of a logit's bits as they are, which takes 13 instructions for
// two of them (21 with the values in their order; counting is bound by them,
// not by its atomics).  Thread t has the t-th block from the largest values
// down: positive ones from their end on.  A row with more than 65535 logits of
// one value is counted in 32 bits instead, in windows of 32 values a thread.
constexpr int kPositive = kSampleThreads / 2;  // blocks of positive values
constexpr int kWindow = 32 * kSampleThreads;  // 128 KiB
struct SampleShared {
  uint32_t count[kWindow];
  double mass[kSampleThreads];  // sums up to and with the thread's values
  uint32_t held[kSampleThreads];
  double root[32];              // 2^(i / 32)
  double wave_mass[kSampleWaves];
  uint32_t waves[kSampleWaves], more[kSampleWaves];
  int first[kSampleWaves];
  double answer_mass;
  int64_t answer_n, below;
  int answer_key;
  uint32_t answer_in, found;
  uint32_t lowest;  // logits of the type's lowest value
};

// e^d for d <= 0 in 64 bits: 2^(n/32) from a table times a polynomial of what
// is left, |r| <= ln 2 / 64 (P. T. P. Tang, "Table-driven implementation of the
// exponential function in IEEE floating-point arithmetic", 1989).
__device__ __forceinline__ double sample_exp(double d, const double *root) {
  if (!(d >= -744.0)) return 0.0;  // a NaN too: no share
  const double n = __builtin_rint(d * 46.166241308446828384);         // 32 / ln 2
  double r = __builtin_fma(n, -0x1.62e42fefp-6, d);                   // ln 2 / 32: its first 33 bits,
  r = __builtin_fma(n, -0x1.473de6af278edp-39, r);                    // and the rest
  double p = 1.0 / 720.0;  // up to r^6: 2^-58 of the result (to r^5, 2^-49, which a block's sum takes to the 63rd power)
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  const int i = (int)n;
  const double f = root[i & 31];
  return __builtin_ldexp(__builtin_fma(f * r, p, f), i >> 5);
}

// A logit's place in the order of its type's values is its magnitude's bits, or
// less them; minus zero has zero's.  Two logits a dword.
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ i16x2 sample_keys(uint32_t two) {
  const i16x2 v = __builtin_bit_cast(i16x2, two), sign = v >> 15;
  return (__builtin_bit_cast(i16x2, two & 0x7FFF7FFFu) ^ sign) - sign;
}
template <typename T>
__device__ __forceinline__ double sample_value(int key) {
  return (double)widen<T>((uint16_t)(key < 0 ? 0x8000 - key : key));
}
// minus infinity's, which is the lowest where there is no NaN
template <typename T>
constexpr int kLowestKey = std::is_same_v<T, _Float16> ? -0x7C00 : -0x7F80;

// Masks are often that value instead of minus infinity: a vocabulary's worth of it
// is counted in 32 bits, and not by atomics that all meet on one dword (rows of
// 131072 and 50021, all but ten: 19 and 21 us, 275 and 60 as other values).  The last
// of its block:
template <typename T>
constexpr int kLowestBlock = kPositive + (-kLowestKey<T> - 1) / 64;
static_assert((-kLowestKey<_Float16> - 1) % 64 == 63 && (-kLowestKey<__bf16> - 1) % 64 == 63, "");

struct SampleSettings {
  float u, top_p, min_p;
  int k;
};

template <typename T>
struct Sampler {
  SampleShared &s;
  const uint16_t *row;
  int V, tid, lane, wave;
  int top;                // the largest logit's key
  double largest, slope;  // its value; 1 / temperature
  int window;             // which one is counted
  uint32_t lowest;        // logits of the type's lowest value, of a packed row

  // Eight logits from an index on; minus infinity past the row's end.
  __device__ __forceinline__ u32x4 eight(int base) const {
    constexpr uint32_t LOW = std::is_same_v<T, _Float16> ? 0xFC00FC00u : 0xFF80FF80u;
    u32x4 v = {LOW, LOW, LOW, LOW};
    if (base + 8 <= V) {
      v = *reinterpret_cast<const u32x4_any *>(row + base);
    } else if (base < V) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (base + e < V) v[e / 2] = e % 2 ? (v[e / 2] & 0xFFFFu) | (uint32_t)row[base + e] << 16 : (v[e / 2] & 0xFFFF0000u) | row[base + e];
    }
    return v;
  }
  // f of eight logits, over a run of the row by threads `first`, first + step, ..; U loads are on the way at once,
  // without a branch between them.  Where f returns true, `rare` gets each two of them again and the first one's
  // index: its code is there once, and not between the steps that are taken every time.
  template <int U, typename F, typename R>
  __device__ __forceinline__ void each(int from, int to, int first, int step, F &&f, R &&rare) const {
    const int n = (to - from) / 8;
    uint32_t again = 0;
#pragma unroll 1
    for (int i0 = first; i0 <= n; i0 += U * step) {
      u32x4 v[U];
      if (i0 < n) {
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = *reinterpret_cast<const u32x4_any *>(row + from + (i0 + i * step < n ? i0 + i * step : i0) * 8);
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (i0 + i * step < n && f(v[i])) again |= 1u << i;
      }
      if (from + n * 8 < to && (unsigned)(n - i0) % step == 0 && (n - i0) / step < U) again |= 1u << (n - i0) / step;
      while (again) {
        const int base = from + (i0 + __builtin_ctz(again) * step) * 8;
        again &= again - 1;
        u32x4 w = eight(base);
#pragma unroll 1
        for (int d = 0; d < 4; ++d) {
          rare(w[0], base + 2 * d);
          w = u32x4{w[1], w[2], w[3], 0u};
        }
      }
    }
  }

  __device__ __forceinline__ double share(int key) const {
    if (key >= top) return 1.0;  // (above it there is no logit)
    const double d = (sample_value<T>(key) - largest) * slope;
    return d < 0.0 ? sample_exp(d, s.root) : d == 0.0 ? 1.0 : 0.0;  // a NaN: an infinite largest one, at an infinite temperature
  }
  // How values lie in the counts: in blocks of `bins` a thread, from `start` down in a window, else from the largest
  // there is, with zero in two places, the second one empty.
  bool packed;
  int bins, start;
  __device__ __forceinline__ int key_at(int block, int i) const {
    return start - block * bins - i + (packed && block >= kPositive);
  }
  __device__ __forceinline__ uint32_t count_at(int block, int i) const {
    const int of = packed && block < kPositive ? block ^ (kPositive - 1) : block;
    const uint32_t v = s.count[of * 32 + ((i ^ block) & 31)];
    if (packed && block == kLowestBlock<T> && i == 63) return lowest;
    return packed ? v >> (((i >> 5) ^ (block < kPositive)) << 4) & 0xFFFFu : v;
  }

  __device__ __forceinline__ void clear() const {
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<u32x4 *>(s.count + (i * kSampleThreads + tid) * 4) = u32x4{0u, 0u, 0u, 0u};
  }

  // Counts the whole row, whose counts are clear, in 16 bits, from the largest
  // key there is down, and finds the largest logit; false if there is nothing to
  // take, or a NaN.  Minus infinity, which may be most of a row, is left out.
  __device__ __forceinline__ bool count_all() {
    packed = true;
    window = 0;
    bins = 64;
    start = 0x7FFF;
    if (tid == 0) s.found = s.lowest = 0;
    __syncthreads();
    constexpr uint32_t LOW = 0x10000u - (0x8000u + kLowestKey<T>);  // minus infinity's bits; above them, NaN with a sign
    uint64_t aside = 0;  // how many are not counted in place, and of these, times 2^32, the lowest values
    auto count = [&](uint32_t two, bool both, bool lo, bool hi) {
      // dwords p / 64 * 32 + (p ^ p / 64) % 32; 16 for the second half
      const u16x2 p = __builtin_bit_cast(u16x2, two);
      const uint32_t mixed = __builtin_bit_cast(uint32_t, p ^ (p >> 6)), half = __builtin_bit_cast(uint32_t, p >> 1);
      const uint32_t word = (mixed & 0x001F001Fu) | (half & ~0x001F001Fu), shift = half & 0x00100010u;
      if (both || lo) atomicAdd(&s.count[word & 0xFFFFu], 1u << (shift & 31u));
      if (both || hi) atomicAdd(&s.count[word >> 16], 1u << (shift >> 16));
    };
    each<4>(0, V, tid, kSampleThreads,
            [&](const u32x4 &v) {
              u16x2 most = {0, 0}, least = {0xFFFF, 0xFFFF};
#pragma unroll
              for (int d = 0; d < 4; ++d) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, +v[d]));
              if (most[0] < LOW - 1 && most[1] < LOW - 1) {
#pragma unroll
                for (int d = 0; d < 4; ++d) count(v[d], true, true, true);
                return false;
              }
              // all of them minus infinity, or the lowest value?
#pragma unroll
              for (int d = 0; d < 4; ++d) least = __builtin_elementwise_min(least, __builtin_bit_cast(u16x2, +v[d]));
              const uint32_t all = most[0];
              if (most[1] != all || least[0] != all || least[1] != all || all > LOW) return true;
              aside += all < LOW ? 8ull << 32 | 8 : 8;
              return false;
            },
            [&](uint32_t two, int) {
              const uint32_t lo = two & 0xFFFFu, hi = two >> 16;
              count(two, false, lo < LOW - 1, hi < LOW - 1);
              aside += (lo >= LOW - 1) + (hi >= LOW - 1) + ((uint64_t)((lo == LOW - 1) + (hi == LOW - 1)) << 32);
              if (lo > LOW || hi > LOW) s.found = 1;
            });
    uint32_t low = (uint32_t)(aside >> 32);
    if (__any(low != 0)) {
      low = wave_scan(low);
      if (lane == 63) atomicAdd(&s.lowest, low);
    }
    __syncthreads();
    if (tid == 0) {  // minus zero is zero
      constexpr int minus = kPositive * 32;
      const uint32_t zeros = s.count[minus] & 0xFFFFu;
      s.count[minus] -= zeros;
      s.count[0] += zeros;
    }
    __syncthreads();
    const uint32_t *mine = s.count + (tid < kPositive ? tid ^ (kPositive - 1) : tid) * 32;
    uint32_t n = 0;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
      const uint32_t c = mine[(i ^ tid) & 31];
      n += (c & 0xFFFFu) + (c >> 16);
    }
    const uint32_t lost = (tid == 0 ? ((uint32_t)V + 7) & ~7u : 0u) - (uint32_t)aside - n;  // together nothing
    lowest = (uint32_t)__builtin_amdgcn_readfirstlane((int)s.lowest);
    if (tid == kLowestBlock<T>) n += lowest;
    const uint64_t here = __ballot(n != 0);
    if (lane == 0) s.first[wave] = here ? wave * 64 + __builtin_ctzll(here) : kSampleThreads;
    __syncthreads();
    int g = kSampleThreads;
#pragma unroll
    for (int i = 0; i < kSampleWaves; ++i) g = s.first[i] < g ? s.first[i] : g;
    g = __builtin_amdgcn_readfirstlane(g);
    const bool none = g == kSampleThreads;  // nothing, or a multiple of 2^16 of one value that left no carry
    if (s.found || (none && V <= 0xFFFF)) return false;
    const uint64_t held = none ? 1 : __ballot(count_at(g, lane) != 0);
    const int j0 = (int)__builtin_ctzll(held);  // (if a count ran over, another key's: found below; infinity's, a NaN's)
    top = key_at(g, j0);
    largest = sample_value<T>(top);

    // The shares of a block's values, equally far apart since binades begin at
    // multiples of 64, as a polynomial of their ratio, a count and a product each.
    double m = 0.0;
    if (__any(n != 0)) {
      const int key = key_at(tid, 0);
      const double r = sample_exp((sample_value<T>(key - 1) - sample_value<T>(key)) * slope, s.root);
      const int near = tid < kPositive ? 16 : 0;  // the first 32 values' counts
      double far = 0.0, r32 = r;
      uint32_t last = tid == kLowestBlock<T> ? lowest : 0;  // more of the last value
#pragma unroll 8
      for (int i = 31; i >= 0; --i) {
        const uint32_t v = mine[(i ^ tid) & 31], c = __builtin_rotateright32(v, near);
        m = __builtin_fma(m, r, (double)(c & 0xFFFFu));
        far = __builtin_fma(far, r, (double)((c >> 16) + last));
        last = 0;
      }
#pragma unroll
      for (int i = 0; i < 5; ++i) r32 *= r32;
      m = __builtin_fma(far, r32, m);
      // (the block of the largest logit may begin above it)
      const double d = (sample_value<T>(key) - largest) * slope;
      m = n ? m * (d == 0.0 ? 1.0 : sample_exp(d, s.root)) : 0.0;
      if (wave == g >> 6 && !(read_lane(d, g & 63) < 600.0)) {  // where that leaves the range: one value a lane
        const uint32_t c = count_at(g, lane);
        const double of_g = read_lane(wave_scan(c ? (double)c * share(key_at(g, lane)) : 0.0), 63);
        if (tid == g) m = of_g;
      }
    }
    // A 16-bit count that runs over takes 2^16 from itself and adds at most one elsewhere: the counts' sum is then too small,
    // modulo 2^32 too, since a row has fewer logits.
    add_up(n, m, lost);
    if (V > 0xFFFF && (none || s.below != 0)) {
      packed = false;
      return find_top();
    }
    return top <= -kLowestKey<T>;  // else a NaN
  }

  // The largest logit by reading the row; false as count_all.
  __device__ __forceinline__ bool find_top() {
    i16x2 most = {-0x7FFF, -0x7FFF};
    u16x2 magnitude = {0, 0};
    auto two = [&](uint32_t v) {
      most = __builtin_elementwise_max(most, sample_keys(v));
      magnitude = __builtin_elementwise_max(magnitude, __builtin_bit_cast(u16x2, v & 0x7FFF7FFFu));
    };
    each<4>(0, V, tid, kSampleThreads,
            [&](const u32x4 &v) {
#pragma unroll
              for (int d = 0; d < 4; ++d) two(v[d]);
              return false;
            },
            [&](uint32_t v, int) { two(v); });
    int t = most[0] > most[1] ? most[0] : most[1];
    if ((magnitude[0] > magnitude[1] ? magnitude[0] : magnitude[1]) > -kLowestKey<T>) t = 0x10000;  // a NaN
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      const int o = __shfl_xor(t, d);
      t = o > t ? o : t;
    }
    __syncthreads();
    if (lane == 0) s.first[wave] = t;
    __syncthreads();
    for (int w = 0; w < kSampleWaves; ++w) t = s.first[w] > t ? s.first[w] : t;
    top = __builtin_amdgcn_readfirstlane(t);
    largest = sample_value<T>(top);
    return top <= 0x7FFF && top > kLowestKey<T>;
  }

  __device__ __forceinline__ void add_up(uint32_t n, double m, uint32_t below) {
    const uint32_t with = wave_scan(n);
    const double with_m = wave_scan(m);
    below = wave_scan(below);
    if (lane == 63) {
      s.waves[wave] = with;
      s.wave_mass[wave] = with_m;
      s.more[wave] = below;
    }
    __syncthreads();
    const int i = lane < kSampleWaves ? lane : kSampleWaves - 1;
    const uint32_t upto = wave_scan(s.waves[i]);
    const double upto_m = wave_scan(s.wave_mass[i]);
    int64_t more = 0;
    if (wave == 0) {
#pragma unroll
      for (int w = 0; w < kSampleWaves; ++w) more += s.more[w];
    }
    const int last = wave > 0 ? wave - 1 : 0;
    const uint32_t before = wave > 0 ? (uint32_t)__builtin_amdgcn_readlane((int)upto, last) : 0u;
    const double before_m = wave > 0 ? read_lane(upto_m, last) : 0.0;
    s.held[tid] = before + with;
    s.mass[tid] = before_m + with_m;
    if (tid == 0) s.below = packed ? (int64_t)(uint32_t)more : more;
    __syncthreads();
  }

  // Counts window w in 32 bits.
  __device__ __forceinline__ void count_window(int w) {
    __syncthreads();
    clear();
    packed = false;
    window = w;
    bins = 32;
    start = top - w * kWindow;
    __syncthreads();
    const uint32_t skip = (uint32_t)w * kWindow, all = (uint32_t)(top - kLowestKey<T>) - skip;
    const uint32_t inside = all < (uint32_t)kWindow ? all : (uint32_t)kWindow;
    const i16x2 tops = {(int16_t)top, (int16_t)top};
    uint32_t below = 0;
    auto count = [&](uint32_t v) {
      const uint32_t two = __builtin_bit_cast(uint32_t, tops - sample_keys(v));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t i = (h ? two >> 16 : two & 0xFFFFu) - skip;
        if (i < inside)
          atomicAdd(&s.count[(i & ~31u) | ((i ^ i >> 5) & 31u)], 1u);
        else if (i < all)  // (places of the windows before this one have wrapped to the far end)
          ++below;
      }
    };
    each<4>(0, V, tid, kSampleThreads,
            [&](const u32x4 &v) {
#pragma unroll
              for (int d = 0; d < 4; ++d) count(v[d]);
              return false;
            },
            [&](uint32_t v, int) { count(v); });
    __syncthreads();
    uint32_t n = 0;
    double m = 0.0;
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
      const uint32_t c = count_at(tid, i);
      if (c) {
        n += c;
        m = __builtin_fma((double)c, share(key_at(tid, i)), m);
      }
    }
    add_up(n, m, below);
  }

  struct Found {
    int64_t n;    // tokens up to and with it
    double mass;  // their sum
    int key;
    uint32_t in;  // which of its value's tokens it is, from 1
  };

  enum class What { Count, Reaches, Passes, Under };

  // In the counted window, after n0 tokens of sum m0: the first token with
  // n >= want, with S_n >= mass, with S_n > mass, or the last before the first
  // with e_i < mass.  False, with what the window holds added, if there is none.
  // For one wave alone.
  __device__ __forceinline__ bool search(What what, int64_t want, double mass, Found *f) const {
    const int64_t n0 = f->n;
    const double m0 = f->mass;
    auto there = [&](int64_t n, double m, int key) {
      if (what == What::Count) return n0 + n >= want;
      if (what == What::Reaches) return m0 + m >= mass;
      if (what == What::Passes) return m0 + m > mass;
      return key <= kLowestKey<T> || share(key) < mass;
    };
    // blocks by sixteens, one of sixteen, one of its values
    auto block_there = [&](int g) { return there(s.held[g], s.mass[g], key_at(g, bins - 1)); };
    uint64_t hit = __ballot(block_there(lane * 16 + 15));
    if (hit == 0) {
      f->n = n0 + s.held[kSampleThreads - 1];
      f->mass = m0 + s.mass[kSampleThreads - 1];
      f->in = 0;
      return false;
    }
    const int some = __builtin_ctzll(hit) * 16;
    hit = __ballot(lane < 16 && block_there(some + (lane & 15)));
    const int g = some + (hit ? __builtin_ctzll(hit) : 15);
    const int key = key_at(g, lane);
    const uint32_t c = lane < bins ? count_at(g, lane) : 0u;
    const double e = c ? share(key) : 0.0;
    const uint32_t n = wave_scan(c);
    const double m = wave_scan((double)c * e);
    const int64_t bn = g ? s.held[g - 1] : 0;
    const double bm = g ? s.mass[g - 1] : 0.0;
    hit = __ballot(lane < bins && there(bn + n, bm + m, key) && (c != 0 || what == What::Under));
    // the block's sum and its values' may round to either side of the border: its last value then
    const uint64_t any = __ballot(c != 0);
    const int at = hit ? __builtin_ctzll(hit) : any ? 63 - __builtin_clzll(any) : bins - 1;
    const uint32_t count = (uint32_t)__builtin_amdgcn_readlane((int)c, at);
    const int64_t nb = n0 + bn + (uint32_t)__builtin_amdgcn_readlane((int)n, at) - count;  // tokens of the values before
    const double one = read_lane(e, at);
    const double mb = m0 + bm + read_lane(m, at) - (double)count * one;
    uint32_t in = count;
    if (what == What::Count) {
      in = (uint32_t)(want - nb);
    } else if (what == What::Under) {
      in = 0;
    } else if (one > 0.0) {
      const double k = (mass - mb) / one;
      const double r = what == What::Reaches ? ceil(k) : floor(k) + 1.0;
      in = r < 1.0 ? 1u : r > (double)count ? count : (uint32_t)r;
    }
    *f = Found{nb + in, mb + (double)in * one, key_at(g, at), in};
    return true;
  }

  // What top_k leaves, the whole row without it; what top_p, and min_p, leave of
  // that; the token; and if rounding put it past what is kept, the last of that.
  template <typename F>
  __device__ __forceinline__ static Found choose(const SampleSettings &set, F &&find) {
    Found kept{0, 0.0, 0, 0}, f{0, 0.0, 0, 0};
    double all = 0.0;
#pragma unroll 1
    for (int step = 0; step < 5; ++step) {
      if (step == 1 && !(set.top_p < 1.0f)) continue;
      if (step == 2 && !(set.min_p > 0.0f)) continue;
      if (step == 4 && f.in != 0 && f.n <= kept.n) break;
      const What what = step == 1 ? What::Reaches : step == 2 ? What::Under : step == 3 ? What::Passes : What::Count;
      const int64_t want = step == 4 ? kept.n : set.k > 0 ? set.k : INT64_MAX;
      f = find(what, want, step == 1 ? (double)set.top_p * all : step == 2 ? (double)set.min_p : (double)set.u * kept.mass);
      if (step == 0) all = f.mass;
      if (step == 0 || (step < 3 && f.n < kept.n)) kept = f;
    }
    return f;
  }

  // The same over all windows, for the whole workgroup.
  __device__ __forceinline__ Found find(What what, int64_t want, double mass) {
    Found f{0, 0.0, 0, 0};
    for (int w = 0;; ++w) {
      if (w != window) count_window(w);
      if (wave == 0) {
        const bool found = search(what, want, mass, &f);
        if (lane == 0) {
          s.answer_n = f.n;
          s.answer_mass = f.mass;
          s.answer_key = f.key;
          s.answer_in = f.in;
          s.found = found;
        }
      }
      __syncthreads();
      f = Found{s.answer_n, s.answer_mass, s.answer_key, s.answer_in};
      const bool over = s.found != 0 || s.below == 0;
      __syncthreads();
      if (over) return f;
    }
  }

  // The index of the `which`-th logit with a key, from 1.  The logits with it are
  // listed in the order of their atomics, and the one that has which - 1 of them
  // before it is taken; more than a thread has room for are counted by runs of the row
  // instead.
  __device__ __forceinline__ int place_of(int key, uint32_t which) {
    uint32_t *list = s.count;  // done with
    const uint32_t bits = (uint32_t)(key < 0 ? 0x8000 - key : key) * 0x10001u;
    const uint32_t mask = key == 0 ? 0x7FFF7FFFu : 0xFFFFFFFFu;  // either zero
    __syncthreads();
    if (tid == 0) s.found = 0;
    __syncthreads();
    each<4>(0, V, tid, kSampleThreads,
            [&](const u32x4 &v) {
              u16x2 least = {0xFFFF, 0xFFFF};
#pragma unroll
              for (int d = 0; d < 4; ++d) least = __builtin_elementwise_min(least, __builtin_bit_cast(u16x2, (v[d] ^ bits) & mask));
              return least[0] == 0 || least[1] == 0;
            },
            [&](uint32_t two, int base) {
              const uint32_t t = (two ^ bits) & mask;
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if ((t >> (16 * e) & 0xFFFFu) == 0 && base + e < V) {
                  const uint32_t at = atomicAdd(&s.found, 1u);
                  if (at < kSampleThreads) list[at] = (uint32_t)(base + e);
                }
            });
    __syncthreads();
    const uint32_t n = s.found;
    if (n <= kSampleThreads) {
      if (n == 1) return (int)list[0];
      if (tid < (int)n) {
        const uint32_t mine = list[tid];
        uint32_t before = 0;
        for (uint32_t i = 0; i < n; ++i) before += list[i] < mine;
        if (before + 1 == which) s.answer_n = mine;
      }
      __syncthreads();
      return (int)s.answer_n;
    }
    const int run = (V + kSampleWaves * 512 - 1) / (kSampleWaves * 512) * 512;  // a wave's, below 2^27
    const int from = wave * run, to = V - from < run ? V : from + run;
    auto matches = [&](uint32_t two, int base, int e) {
      return (((two ^ bits) & mask) >> (16 * e) & 0xFFFFu) == 0 && base + e < to;
    };
    uint32_t ours = 0;
    auto count = [&](uint32_t two, int base) { ours += matches(two, base, 0) + matches(two, base, 1); };
    each<4>(from, to, lane, 64,
            [&](const u32x4 &v) {
#pragma unroll
              for (int d = 0; d < 4; ++d) count(v[d], from);
              return false;
            },
            [&](uint32_t two, int base) { count(two, base); });
    ours = wave_scan(ours);
    if (lane == 63) s.waves[wave] = ours;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < wave; ++w) before += s.waves[w];
    if (before < which && which <= before + s.waves[wave]) {
      for (int base = from + lane * 8; base - lane * 8 < to; base += 512) {
        const u32x4 v = eight(base);
        uint32_t mine = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) mine += matches(v[e / 2], base + (e & ~1), e % 2);
        const uint32_t with = wave_scan(mine);
        uint32_t at = before + with - mine;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (matches(v[e / 2], base + (e & ~1), e % 2) && ++at == which) s.answer_n = base + e;
        before += (uint32_t)__shfl((int)with, 63);
      }
    }
    __syncthreads();
    return (int)s.answer_n;
  }
};

// A row whose counts do not fit 16 bits, for the whole workgroup; a function of
// its own, so that its registers are not the other rows' too.
template <typename T>
__device__ __attribute__((noinline)) void sample_wide(SampleShared &s, const uint16_t *logits, int V, int top, double slope,
                                                      SampleSettings set) {
  const int tid = threadIdx.x;
  Sampler<T> row{s, logits, V, tid, tid & 63, tid >> 6, top, sample_value<T>(top), slope, -1, 0, false, 0, 0};
  const auto f = row.choose(set, [&](auto what, int64_t want, double mass) { return row.find(what, want, mass); });
  if (tid == 0) {
    s.answer_key = f.key;
    s.answer_in = f.in;
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kSampleThreads) sample_kernel(SampleArgs a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  SampleShared &s = *reinterpret_cast<SampleShared *>(smem);
  if (threadIdx.x < 32) s.root[threadIdx.x] = exp2((double)threadIdx.x / 32.0);
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    // What follows from these is worked out for every row: ahead of the loop, which most workgroups run through once, it
    // would take more vector registers than there are (26.6 us with their spills, 21.8 without, 256 rows of 50021).
    int tid = threadIdx.x, V = a.V;
    asm volatile("" : "+v"(tid), "+s"(V));
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    auto at = [&](int bit) { return a.shared & bit ? 0 : m; };
    const float u = a.u[m];
    const float t = a.temperature ? a.temperature[at(PGEMM_SAMPLE_TEMPERATURE)] : 1.0f;
    const int k = a.top_k ? a.top_k[at(PGEMM_SAMPLE_TOP_K)] : 0;
    const float top_p = a.top_p ? a.top_p[at(PGEMM_SAMPLE_TOP_P)] : 1.0f;
    const float min_p = a.min_p ? a.min_p[at(PGEMM_SAMPLE_MIN_P)] : 0.0f;

    Sampler<T> row{s, a.logits + m * V, V, tid, lane, wave, 0, 0.0, 1.0, -1, 0, false, 0, 0};
    const bool first = t == 0.0f || top_p <= 0.0f || min_p > 1.0f || k == 1;  // nothing to choose
    row.slope = 1.0 / (double)t;
    bool good = t >= 0.0f && top_p == top_p && min_p == min_p && u == u;
    if (good) {
      if (first) {
        good = row.find_top();
      } else {
        row.clear();
        good = row.count_all();
      }
    }
    if (!good) {
      if (tid == 0) a.token[m] = -1;
      __syncthreads();
      continue;
    }
    const SampleSettings set{u > 0.0f ? u : 0.0f, top_p, min_p, k};
    int key = row.top;
    uint32_t in = 1;
    if (!first) {
      typename Sampler<T>::Found f{0, 0.0, 0, 0};
      if (row.packed) {  // one window holds the row
        if (wave == 0) {
          f = row.choose(set, [&](auto what, int64_t want, double mass) __attribute__((always_inline)) {
            typename Sampler<T>::Found g{0, 0.0, 0, 0};
            row.search(what, want, mass, &g);
            return g;
          });
          if (lane == 0) {
            s.answer_key = f.key;
            s.answer_in = f.in;
          }
        }
        __syncthreads();
      } else {
        sample_wide<T>(s, row.row, row.V, row.top, row.slope, set);
      }
      key = s.answer_key;
      in = s.answer_in;
    }
    const int place = row.place_of(key, in);
    if (tid == 0) a.token[m] = place;
    __syncthreads();
  }
}

namespace launch_detail {

template <typename T>
pgemm_status sample_rows(const SampleCall &c) {
  static std::atomic<uint64_t> lds_set{0};
  auto kern = sample_kernel<T>;
  pgemm_status st = allow_lds(kern, sizeof(SampleShared), c.dev, lds_set);
  if (st != PGEMM_OK) return st;
  SampleArgs a{c.logits, c.u, c.temperature, c.top_k, c.top_p, c.min_p, c.token, c.M, (int)c.V, c.shared};
  const unsigned grid = (unsigned)(c.M < 65536 ? c.M : 65536);
  hipLaunchKernelGGL(kern, dim3(grid), dim3(kSampleThreads), sizeof(SampleShared), c.stream, a);
  return launched();
}

}  // namespace launch_detail
}  // namespace pgemm
