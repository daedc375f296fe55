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
// atomics, and all sums are in 64 bits.  LDS holds the counts of kWindow values
// in order, from the largest down; rows that reach further take the next window.
#pragma once

#include "fused_launch.hpp"
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
constexpr int kSampleGroups = 576;                 // of 64 values each
constexpr int kWindow = kSampleGroups * 64;        // 144 KiB of counts
struct SampleShared {
  uint32_t count[kWindow];
  double mass[kSampleGroups];   // sums up to and with the group
  uint32_t held[kSampleGroups];
  uint32_t waves[kSampleWaves], more[kSampleWaves];
  double answer_mass;
  int64_t answer_n, below;
  uint32_t answer_key, answer_in;
};

// A logit's place in the order of its type's values: 16 bits, 0 for a NaN.
template <typename T>
__device__ __forceinline__ uint32_t sample_key(uint32_t bits) {
  constexpr uint32_t INF = std::is_same_v<T, _Float16> ? 0x7C00u : 0x7F80u;
  if ((bits & 0x7FFFu) > INF) return 0;
  if (bits == 0x8000u) bits = 0;
  return bits & 0x8000u ? 0xFFFFu - bits : bits | 0x8000u;
}
template <typename T>
__device__ __forceinline__ double sample_value(uint32_t key) {
  const uint32_t bits = key & 0x8000u ? key & 0x7FFFu : 0xFFFFu - key;
  return (double)widen<T>((uint16_t)bits);
}
// minus infinity's
template <typename T>
constexpr uint32_t kLowestKey = std::is_same_v<T, _Float16> ? 0xFFFFu - 0xFC00u : 0xFFFFu - 0xFF80u;

template <typename T>
struct Sampler {
  SampleShared &s;
  const uint16_t *row;
  int V, tid, lane, wave;
  uint32_t top;      // the largest logit's key
  double largest, slope;  // its value; 1 / temperature
  int window;        // which one is counted

  // f(key, index) of all logits, 16 bytes a thread at a time.
  template <typename F>
  __device__ __forceinline__ void each(F &&f) const {
    for (int base = tid * 8; base < V; base += kSampleThreads * 8) {
      if (base + 8 <= V) {
        const u32x4 v = *reinterpret_cast<const u32x4_any *>(row + base);
#pragma unroll
        for (int e = 0; e < 8; ++e) f(sample_key<T>((v[e / 2] >> (16 * (e % 2))) & 0xFFFFu), base + e);
      } else {
        for (int e = base; e < V; ++e) f(sample_key<T>(row[e]), e);
      }
    }
  }

  __device__ __forceinline__ double share(uint32_t key) const {
    const double v = sample_value<T>(key);
    if (v == largest) return 1.0;
    const double d = (v - largest) * slope;
    return d < 0.0 ? exp(d) : d == 0.0 ? 1.0 : 0.0;  // a NaN: an infinite largest one, at an infinite temperature
  }
  // the key of place i of the counted window; negative: past the last value
  __device__ __forceinline__ int key_at(int i) const { return (int)top - window * kWindow - i; }

  // Counts window w and adds the shares of its groups up.
  __device__ __forceinline__ void count(int w) {
    window = w;
    __syncthreads();
    for (int i = tid; i < kWindow; i += kSampleThreads) s.count[i] = 0;
    if (tid == 0) s.below = 0;
    __syncthreads();
    const int first = (int)top - w * kWindow;
    uint32_t below = 0;
    each([&](uint32_t key, int) {
      const int i = first - (int)key;
      if (key > kLowestKey<T> && i >= 0) {
        if (i < kWindow)
          atomicAdd(&s.count[i], 1u);
        else
          ++below;
      }
    });
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) below += (uint32_t)__shfl_xor((int)below, d);
    if (lane == 0) s.more[wave] = below;
    __syncthreads();
    for (int g = wave; g < kSampleGroups; g += kSampleWaves) {
      uint32_t n = s.count[g * 64 + lane];
      double m = 0.0;
      if (__any(n != 0)) m = n ? (double)n * share((uint32_t)key_at(g * 64 + lane)) : 0.0;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) {
        n += (uint32_t)__shfl_xor((int)n, d);
        m += __shfl_xor(m, d);
      }
      if (lane == 0) {
        s.held[g] = n;
        s.mass[g] = m;
      }
    }
    __syncthreads();
    if (wave == 0) {
      constexpr int PER = kSampleGroups / 64;
      uint32_t n = 0;
      double m = 0.0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        n += s.held[lane * PER + i];
        m += s.mass[lane * PER + i];
      }
      uint32_t before = n;
      double before_m = m;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t a = (uint32_t)__shfl_up((int)before, d);
        const double b = __shfl_up(before_m, d);
        if (lane >= d) {
          before += a;
          before_m += b;
        }
      }
      n = before - n;
      m = __shfl_up(before_m, 1);
      if (lane == 0) m = 0.0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        n += s.held[lane * PER + i];
        m += s.mass[lane * PER + i];
        s.held[lane * PER + i] = n;
        s.mass[lane * PER + i] = m;
      }
      if (lane == 0) {
        int64_t all = 0;
        for (int i = 0; i < kSampleWaves; ++i) all += s.more[i];
        s.below = all;
      }
    }
    __syncthreads();
  }

  struct Found {
    int64_t n;    // tokens up to and with it
    double mass;  // their sum
    uint32_t key;
    uint32_t in;  // which of its value's tokens it is, from 1
  };

  enum class What { Count, Reaches, Passes, Under };

  // The first token with n >= count, with S_n >= mass, with S_n > mass, or the
  // last before the first with e_i < mass; the row's last one if there is none.
  template <What W>
  __device__ __forceinline__ Found find(int64_t want, double mass) {
    int64_t n0 = 0;
    double m0 = 0.0;
    for (int w = 0;; ++w) {
      if (w != window) count(w);
      if (wave == 0) {
        auto there = [&](int64_t n, double m, int place) {
          if (W == What::Count) return n0 + n >= want;
          if (W == What::Reaches) return m0 + m >= mass;
          if (W == What::Passes) return m0 + m > mass;
          const int key = key_at(place);
          return key <= (int)kLowestKey<T> || share((uint32_t)key) < mass;
        };
        int g = -1;
        for (int base = 0; base < kSampleGroups && g < 0; base += 64) {
          const uint64_t hit = __ballot(there(s.held[base + lane], s.mass[base + lane], (base + lane) * 64 + 63));
          if (hit) g = base + __builtin_ctzll(hit);
        }
        Found f{n0 + s.held[kSampleGroups - 1], m0 + s.mass[kSampleGroups - 1], 0, 0};
        if (g >= 0) {
          const uint32_t c = s.count[g * 64 + lane];
          const int key = key_at(g * 64 + lane);
          const double e = c ? share((uint32_t)key) : 0.0;
          uint32_t n = c;
          double m = (double)c * e;
#pragma unroll
          for (int d = 1; d < 64; d <<= 1) {
            const uint32_t a = (uint32_t)__shfl_up((int)n, d);
            const double b = __shfl_up(m, d);
            if (lane >= d) {
              n += a;
              m += b;
            }
          }
          const int64_t bn = g ? s.held[g - 1] : 0;
          const double bm = g ? s.mass[g - 1] : 0.0;
          const uint64_t hit = __ballot(there(bn + n, bm + m, g * 64 + lane) && (c != 0 || W == What::Under));
          // the group's sum and its values' may round to either side of the border: its last value then
          const uint64_t any = __ballot(c != 0);
          const int at = hit ? __builtin_ctzll(hit) : any ? 63 - __builtin_clzll(any) : 63;
          const uint32_t here = (uint32_t)__shfl((int)c, at);
          const int64_t nb = n0 + bn + (uint32_t)__shfl((int)n, at) - here;  // tokens of the values before
          const double one = __shfl(e, at);
          const double mb = m0 + bm + __shfl(m, at) - (double)here * one;
          uint32_t in = here;
          if (W == What::Count) {
            in = (uint32_t)(want - nb);
          } else if (W == What::Under) {
            in = 0;
          } else if (one > 0.0) {
            const double k = (mass - mb) / one;
            const double r = W == What::Reaches ? ceil(k) : floor(k) + 1.0;
            in = r < 1.0 ? 1u : r > (double)here ? here : (uint32_t)r;
          }
          f = Found{nb + in, mb + (double)in * one, (uint32_t)__shfl(key, at), in};
        }
        if (lane == 0) {
          s.answer_n = f.n;
          s.answer_mass = f.mass;
          s.answer_key = f.key;
          s.answer_in = g >= 0 ? f.in + 1 : 0;
        }
      }
      __syncthreads();
      const Found f{s.answer_n, s.answer_mass, s.answer_key, s.answer_in ? s.answer_in - 1 : 0};
      const bool over = s.answer_in != 0 || s.below == 0;
      __syncthreads();
      if (over) return f;
      n0 = f.n;
      m0 = f.mass;
    }
  }

  // The index of the `which`-th logit with a key, from 1.
  __device__ __forceinline__ int place_of(uint32_t key, uint32_t which) {
    const int share = (V + kSampleWaves * 64 - 1) / (kSampleWaves * 64) * 64;  // a wave's run
    const int from = wave * share, to = from + share < V ? from + share : V;
    uint32_t n = 0;
    for (int base = from; base < to; base += 64)
      n += (uint32_t)__popcll(__ballot(base + lane < to && sample_key<T>(row[base + lane]) == key));
    __syncthreads();
    if (lane == 0) s.waves[wave] = n;
    if (tid == 0) s.answer_n = -1;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < wave; ++w) before += s.waves[w];
    if (before < which && which <= before + n) {
      for (int base = from; base < to; base += 64) {
        const bool is = base + lane < to && sample_key<T>(row[base + lane]) == key;
        const uint64_t who = __ballot(is);
        const uint32_t mine = before + (uint32_t)__popcll(who & ((2ull << lane) - 1));
        if (is && mine == which) s.answer_n = base + lane;
        before += (uint32_t)__popcll(who);
      }
    }
    __syncthreads();
    return (int)s.answer_n;
  }
};

template <typename T>
__global__ void __launch_bounds__(kSampleThreads) sample_kernel(SampleArgs a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  SampleShared &s = *reinterpret_cast<SampleShared *>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    auto at = [&](int bit) { return a.shared & bit ? 0 : m; };
    const float u = a.u[m];
    const float t = a.temperature ? a.temperature[at(PGEMM_SAMPLE_TEMPERATURE)] : 1.0f;
    const int k = a.top_k ? a.top_k[at(PGEMM_SAMPLE_TOP_K)] : 0;
    const float top_p = a.top_p ? a.top_p[at(PGEMM_SAMPLE_TOP_P)] : 1.0f;
    const float min_p = a.min_p ? a.min_p[at(PGEMM_SAMPLE_MIN_P)] : 0.0f;

    Sampler<T> row{s, a.logits + m * a.V, a.V, tid, lane, wave, 0, 0.0, 1.0, -1};
    uint32_t top = 0, odd = 0;
    row.each([&](uint32_t key, int) {
      top = key > top ? key : top;
      odd |= key == 0;
    });
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)top, d);
      top = o > top ? o : top;
    }
    __syncthreads();
    if (__any(odd)) top = 0x10000u;
    if (lane == 0) s.waves[wave] = top;
    __syncthreads();
    top = 0;
    for (int w = 0; w < kSampleWaves; ++w) top = s.waves[w] > top ? s.waves[w] : top;
    const bool none = top > 0xFFFFu || top <= kLowestKey<T> || !(t >= 0.0f) || top_p != top_p || min_p != min_p || u != u;
    if (none) {
      if (tid == 0) a.token[m] = -1;
      __syncthreads();
      continue;
    }
    row.top = top;
    row.largest = sample_value<T>(top);
    uint32_t key = top, in = 1;
    if (t > 0.0f && !(top_p <= 0.0f) && !(min_p > 1.0f) && k != 1) {
      row.slope = 1.0 / (double)t;
      using What = typename Sampler<T>::What;
      // what top_k leaves; without it the whole row
      typename Sampler<T>::Found kept = row.template find<What::Count>(k > 0 ? k : INT64_MAX, 0.0);
      const auto last = kept;
      if (top_p < 1.0f) kept = row.template find<What::Reaches>(0, (double)top_p * last.mass);
      if (min_p > 0.0f) {
        const auto f = row.template find<What::Under>(0, (double)min_p);
        if (f.n < kept.n) kept = f;
      }
      const auto f = row.template find<What::Passes>(0, (double)u * kept.mass);
      if (f.in != 0 && f.n <= kept.n) {
        key = f.key;
        in = f.in;
      } else {  // the last that is kept
        const auto e = row.template find<What::Count>(kept.n, 0.0);
        key = e.key;
        in = e.in;
      }
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
