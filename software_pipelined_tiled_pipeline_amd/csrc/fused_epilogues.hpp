// Epilogues of the fused products.  Each gets a wave's settled accumulators:
// lane l, register r of acc[i][j] is row 16 i + l % 16 and column
// 16 j + 4 (l / 16) + r of the wave's block; the ring is free for staging.
#pragma once

#include "fused_gemm.hpp"

namespace pgemm {

constexpr float kLog2e = 1.44269504088896340736f;

// e^x through v_exp_f32 (2^x): the product's rounding costs |x| 2^-24.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// 2^(x log2 e - off), the exponential of a logit from its row's log2 e * reference
__device__ __forceinline__ float exp_from(float x, float off) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(x, kLog2e, -off));
}
// The larger of three in one instruction (a NaN may get lost).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// The gate's activation and its derivative in fp32.  act 0: silu, g s(g);
// act 1: gelu in its tanh form, (1 + tanh y) / 2 = s(2 y).  The derivative's
// polynomial is taken at |g| <= 64 so that its square does not overflow into
// 0 * inf where s (1 - s) has long vanished.
struct Activation {
  float a, d;
};
__device__ __forceinline__ float gate_sigmoid(int act, float g) {
  const float y = act == 0 ? g : 1.5957691216057308f * g * (1.0f + 0.044715f * g * g);
  return __builtin_amdgcn_rcpf(1.0f + fast_exp(-y));
}
__device__ __forceinline__ float activate(int act, float g) { return g * gate_sigmoid(act, g); }
__device__ __forceinline__ Activation activate_slope(int act, float g) {
  const float s = gate_sigmoid(act, g);
  float q = 1.0f;
  if (act != 0) {
    const float c = fminf(fmaxf(g, -64.0f), 64.0f);
    q = 1.5957691216057308f * (1.0f + 0.134145f * c * c);
  }
  return Activation{g * s, s + g * (s * (1.0f - s)) * q};
}

// fp32 of a 16-bit value
template <typename T>
__device__ __forceinline__ float widen(uint16_t v) {
  return (float)__builtin_bit_cast(T, v);
}

// Copies columns [c0, c0 + BN) of a staged tile to out[m0..][n0..], row pitch
// `po`: whole 16-byte pieces wherever they start (an odd pitch leaves them
// at even addresses), single elements at the right edge.  A thread keeps its
// columns and takes eight rows at a time, so that their LDS reads overlap.
template <int BM, int BN, int THREADS>
__device__ __forceinline__ void store_tile(const char *st, int pitch, int c0, uint16_t *out, int64_t po, int M, int N,
                                           int m0, int n0, int tid) {
  constexpr int CH = BN / 8, ROWS = THREADS / CH, PASSES = BM / ROWS;
  constexpr int U = PASSES < 8 ? PASSES : 8;
  static_assert(THREADS % CH == 0 && BM % ROWS == 0 && PASSES % U == 0, "whole passes");
  const int c = tid % CH, r0 = tid / CH, gn = n0 + 8 * c;
  if (gn >= N) return;
  const char *from = st + r0 * pitch + (c0 + 8 * c) * 2;
  uint16_t *to = out + (int64_t)(m0 + r0) * po + gn;
  const int rows = M - m0 - r0;  // inside the matrix, from this thread's first
  for (int p = 0; p < PASSES; p += U) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const u32x4 *>(from + (p + u) * ROWS * pitch);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = (p + u) * ROWS;
      if (row >= rows) continue;
      uint16_t *dst = to + row * po;
      if (gn + 8 <= N) {
        *reinterpret_cast<u32x4_any *>(dst) = v[u];
      } else {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (gn + x < N) dst[x] = (uint16_t)(v[u][x / 2] >> (16 * (x % 2)));
      }
    }
  }
}

// Exponents of the powers of two that an output still has to be multiplied by
// may wait in the output itself: in the first element of each 128 x 128 block
// (DyScale).  A tile's own is read by its workgroup alone, before it stores the
// tile.
constexpr int kSeedStep = 128;  // tiles start at multiples of it
__device__ __forceinline__ float seeded_scale(const uint16_t *out, int64_t po, int m0, int n0) {
  return ldexpf(1.0f, (int16_t)out[(int64_t)m0 * po + n0]);
}

// out = round((sum + acc) * *scale): one product, or the last of several whose
// running sum is kept in fp32 (SumEpi).
struct StoreEpi {
  struct Args {
    uint16_t *out;
    int64_t po;
    const float *scale;  // one device float, or null
    bool seeded;         // the factor is a power of two that waits in out
  };
  template <typename T, class G, class W>
  struct Run {
    // `sum`: null, or what to add, row pitch ps (a multiple of 4)
    __device__ __forceinline__ static void finish(W &w, const Args &e, const FusedProduct &g, char *smem, int m0,
                                                  int n0, int wm, int wn, int lane, int tid, const float *sum, int ps) {
      constexpr int PITCH = Staging<G::BN>::PITCH;
      const float k = e.seeded ? seeded_scale(e.out, e.po, m0, n0) : e.scale ? *e.scale : 1.0f;
      const int lr = wm * G::WM + (lane & 15), lc = wn * G::WN + 4 * (lane >> 4);
#pragma unroll
      for (int i = 0; i < W::TM; ++i)
#pragma unroll
        for (int j = 0; j < W::TN; ++j) {
          f32x4 v = w.acc[i][j];
          const int row = m0 + lr + 16 * i, col = n0 + lc + 16 * j;
          if (sum && row < g.M && col < g.N) v += *reinterpret_cast<const f32x4 *>(sum + (int64_t)row * ps + col);
          *reinterpret_cast<u32x2 *>(smem + (lr + 16 * i) * PITCH + (lc + 16 * j) * 2) =
              Mfma<T>::pack4(v[0] * k, v[1] * k, v[2] * k, v[3] * k);
        }
      __syncthreads();
      store_tile<G::BM, G::BN, G::THREADS>(smem, PITCH, 0, e.out, e.po, g.M, g.N, m0, n0, tid);
    }
    __device__ __forceinline__ void operator()(W &w, const Args &e, const FusedProduct &g, char *smem, int m0, int n0,
                                               int wm, int wn, int lane, int tid) const {
      finish(w, e, g, smem, m0, n0, wm, wn, lane, tid, nullptr, 0);
    }
  };
};

// A sum over several products: the running fp32 sum lives in `sum` (row
// pitch a multiple of 4).  first: nothing to add yet; last: rounds to out.
struct SumEpi {
  struct Args {
    float *sum;
    int ps;
    int first, last;
    StoreEpi::Args out;
  };
  template <typename T, class G, class W>
  struct Run {
    __device__ __forceinline__ void operator()(W &w, const Args &e, const FusedProduct &g, char *smem, int m0, int n0,
                                               int wm, int wn, int lane, int tid) const {
      if (e.last) {
        StoreEpi::Run<T, G, W>::finish(w, e.out, g, smem, m0, n0, wm, wn, lane, tid, e.sum, e.ps);
        return;
      }
#pragma unroll
      for (int i = 0; i < W::TM; ++i) {
        const int row = m0 + wm * G::WM + 16 * i + (lane & 15);
        if (row >= g.M) continue;
        float *rp = e.sum + (int64_t)row * e.ps;
#pragma unroll
        for (int j = 0; j < W::TN; ++j) {
          const int col = n0 + wn * G::WN + 16 * j + 4 * (lane >> 4);
          if (col >= g.N) continue;
          f32x4 v = w.acc[i][j];
          if (!e.first) v += *reinterpret_cast<const f32x4 *>(rp + col);
          *reinterpret_cast<f32x4 *>(rp + col) = v;
        }
      }
    }
  };
};

// A piece of K: the sums in fp32, for join_pieces_kernel.
struct PieceEpi {
  struct Args {
    float *part;  // [pieces][M][pp]
    int pp;       // a multiple of 4
    const uint16_t *seeds;  // null, or the output whose factors are taken here (exactly), and its pitch
    int64_t po;
  };
  template <typename T, class G, class W>
  struct Run {
    __device__ __forceinline__ void operator()(W &w, const Args &e, const FusedProduct &g, char *smem, int m0, int n0,
                                               int wm, int wn, int lane, int tid) const {
      float *part = e.part + (int64_t)g.piece * g.M * e.pp;
      const float k = e.seeds ? seeded_scale(e.seeds, e.po, m0, n0) : 1.0f;
#pragma unroll
      for (int i = 0; i < W::TM; ++i) {
        const int row = m0 + wm * G::WM + 16 * i + (lane & 15);
        if (row >= g.M) continue;
#pragma unroll
        for (int j = 0; j < W::TN; ++j) {
          const int col = n0 + wn * G::WN + 16 * j + 4 * (lane >> 4);
          if (col < g.N) *reinterpret_cast<f32x4 *>(part + (int64_t)row * e.pp + col) = w.acc[i][j] * k;
        }
      }
    }
  };
};

// Gated block: even column blocks of a wave hold the gate, odd ones the up
// projection of the same 16 hidden columns.  h = act(gate) * up; `saved`
// (null: not kept) takes both projections in fp32, per row and group of four
// hidden columns the four gates and then the four ups, for the backward pass.
struct GatedEpi {
  struct Args {
    uint16_t *h;
    float *saved;
    int act;
  };
  template <typename T, class G, class W>
  struct Run {
    __device__ __forceinline__ void operator()(W &w, const Args &e, const FusedProduct &g, char *smem, int m0, int n0,
                                               int wm, int wn, int lane, int tid) const {
      constexpr int ON = G::BN / 2, PITCH = Staging<ON>::PITCH;
      const int r = lane & 15, q = lane >> 4;
      const int64_t ps = (int64_t)((g.N + 3) / 4) * 8;
#pragma unroll
      for (int i = 0; i < W::TM; ++i) {
        const int lrow = wm * G::WM + 16 * i + r;
#pragma unroll
        for (int p = 0; p < W::TN / 2; ++p) {
          const f32x4 ga = w.acc[i][2 * p], up = w.acc[i][2 * p + 1];
          const int lcol = wn * (G::WN / 2) + 16 * p + 4 * q;
          if (e.saved && m0 + lrow < g.M && n0 + lcol < g.N) {
            float *sp = e.saved + (m0 + lrow) * ps + (int64_t)(n0 + lcol) * 2;
            *reinterpret_cast<f32x4 *>(sp) = ga;
            *reinterpret_cast<f32x4 *>(sp + 4) = up;
          }
          f32x4 h;
#pragma unroll
          for (int x = 0; x < 4; ++x) h[x] = activate(e.act, ga[x]) * up[x];
          *reinterpret_cast<u32x2 *>(smem + lrow * PITCH + lcol * 2) = Mfma<T>::pack4(h[0], h[1], h[2], h[3]);
        }
      }
      __syncthreads();
      store_tile<G::BM, ON, G::THREADS>(smem, PITCH, 0, e.h, g.N, g.M, g.N, m0, n0, tid);
    }
  };
};

// The factor of dy = [dh up act'(gate) | dh act(gate)] in f16, where dy is
// rounded to 16 bits between the products: binary16 ends at 65504 and has fewer
// bits below 2^-14, so that a mean loss's dh of 1e-5 cost dW 2.8e-3 instead of
// 2.9e-4, and a dy past its end made dx and dW infinite that were not.
//
// |act'| < 1.13, |act(g)| <= |g|, and |g| and |up| are at most |x's row| |w's row|, so
// no entry passes 1.13 B with B = max |dh| * max |x's row| * max |w's row|.  The factor
// is the power of two that takes B into [2^14, 2^15): no entry overflows, and
// those down to B / 2^29 keep all their bits (a usual one is some 2^10 below B).
// dx and dW are multiplied by its inverse, exactly, before they are rounded.
//
// gated_range_kernel takes the maxima.  Their `parts` wait in rows of dw, and
// the inverse's exponent at the tiles' starts in dx and dw: the workspace has no
// room for them.
struct DyScale {
  const float4 *part;  // max |dh|, and bounds of the squared norms of x's and w's rows
  int parts;           // -1: no factor; 0: the exponent is in dx already
  uint16_t *dx, *dw;
  int64_t rows_x, rows_w, D;

  __device__ __forceinline__ static float4 top(float4 a, float4 b) {
    return make_float4(fmaxf(a.x, b.x), fmaxf(a.y, b.y), fmaxf(a.z, b.z), 0.0f);
  }
  __device__ __forceinline__ static float4 wave_top(float4 t) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) t = top(t, make_float4(__shfl_xor(t.x, d), __shfl_xor(t.y, d), __shfl_xor(t.z, d), 0.0f));
    return t;
  }
  // the inverse's exponent
  __device__ __forceinline__ static int exponent(float4 t) {
    const float bound = t.x * sqrtf(t.y) * sqrtf(t.z);  // at most 2^70
    int e = 15;
    if (bound > 0.0f) frexpf(bound, &e);
    return e - 15;
  }
  // leaves it where the products look for it; `first`, step: which of the starts
  __device__ __forceinline__ void seed(int e, int64_t first, int64_t step) const {
    const int64_t across = (D + kSeedStep - 1) / kSeedStep;
    const int64_t in_x = (rows_x + kSeedStep - 1) / kSeedStep * across, in_w = (rows_w + kSeedStep - 1) / kSeedStep * across;
    for (int64_t i = first; i < in_x + in_w; i += step) {
      const int64_t j = i < in_x ? i : i - in_x;
      (i < in_x ? dx : dw)[j / across * kSeedStep * D + j % across * kSeedStep] = (uint16_t)(int16_t)e;
    }
  }
  // The factor, by every wave of every workgroup of dy's kernel.
  __device__ __forceinline__ float take(int tid, int threads) const {
    if (parts < 0) return 1.0f;
    if (parts == 0) return ldexpf(1.0f, -(int16_t)*dx);
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = tid & 63; i < parts; i += 64) t = top(t, part[i]);
    const int e = exponent(wave_top(t));
    seed(e, (int64_t)blockIdx.x * threads + tid, (int64_t)gridDim.x * threads);
    return ldexpf(1.0f, -e);
  }
};

// The gated block's derivative from recomputed projections: with dh read
// here, dy[m] = [dh up act'(gate) | dh act(gate)], one row of 2 N values.
struct GatedSlopeEpi {
  struct Args {
    const uint16_t *dh;
    uint16_t *dy;
    int64_t py;
    int act;
    DyScale scale;
  };
  template <typename T, class G, class W>
  struct Run {
    __device__ __forceinline__ void operator()(W &w, const Args &e, const FusedProduct &g, char *smem, int m0, int n0,
                                               int wm, int wn, int lane, int tid) const {
      constexpr int ON = G::BN / 2, PITCH = Staging<G::BN>::PITCH;
      const int r = lane & 15, q = lane >> 4;
      const float s = e.scale.take(tid, G::THREADS);
#pragma unroll
      for (int i = 0; i < W::TM; ++i) {
        const int lrow = wm * G::WM + 16 * i + r;
#pragma unroll
        for (int p = 0; p < W::TN / 2; ++p) {
          const f32x4 ga = w.acc[i][2 * p], up = w.acc[i][2 * p + 1];
          const int lcol = wn * (G::WN / 2) + 16 * p + 4 * q;
          const int gm = m0 + lrow, gn = n0 + lcol;
          f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
          if (gm < g.M && gn < g.N) {
            const uint16_t *src = e.dh + (int64_t)gm * g.N + gn;
            if (gn + 4 <= g.N) {
              const u32x2 v = *reinterpret_cast<const u32x2_any *>(src);
#pragma unroll
              for (int x = 0; x < 4; ++x) d[x] = widen<T>((uint16_t)(v[x / 2] >> (16 * (x % 2))));
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (gn + x < g.N) d[x] = widen<T>(src[x]);
            }
          }
          f32x4 dg, du;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const Activation v = activate_slope(e.act, ga[x]);
            dg[x] = d[x] * s * up[x] * v.d;
            du[x] = d[x] * s * v.a;
          }
          char *st = smem + lrow * PITCH + lcol * 2;
          *reinterpret_cast<u32x2 *>(st) = Mfma<T>::pack4(dg[0], dg[1], dg[2], dg[3]);
          *reinterpret_cast<u32x2 *>(st + ON * 2) = Mfma<T>::pack4(du[0], du[1], du[2], du[3]);
        }
      }
      __syncthreads();
      store_tile<G::BM, ON, G::THREADS>(smem, PITCH, 0, e.dy, e.py, g.M, g.N, m0, n0, tid);
      store_tile<G::BM, ON, G::THREADS>(smem, PITCH, ON, e.dy + g.N, e.py, g.M, g.N, m0, n0, tid);
    }
  };
};

// A lane's logits of one row, columns c0 + 16 j + x: those past N, at the
// vocabulary's end, are minus infinity.  (A copy: the accumulators themselves,
// written here, would be spilled all through the K loop.)
template <class G, class W>
struct RowLogits {
  f32x4 v[W::TN];
  __device__ __forceinline__ RowLogits(const W &w, int i, bool edge, int c0, int N) {
#pragma unroll
    for (int j = 0; j < W::TN; ++j) v[j] = w.acc[i][j];
    if (edge) {
#pragma unroll
      for (int j = 0; j < W::TN; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (c0 + 16 * j + x >= N) v[j][x] = -INFINITY;
    }
  }
};

// Softmax statistics of a tile of logits: per row and wave column the
// largest logit and the sum of e^(z - largest), and the target's logit.  A
// tile's 256 values a lane cost 1.5 plain operations and an exponential each;
// what few rows need, the vocabulary's end and the targets, is branched around.
struct LseEpi {
  struct Args {
    float2 *part;  // [tiles_n * WGN][M], of this launch's columns
    float *at;     // [M] the target's logit
    const int64_t *target;
  };
  template <typename T, class G, class W>
  struct Run {
    __device__ __forceinline__ void operator()(W &w, const Args &e, const FusedProduct &g, char *smem, int m0, int n0,
                                               int wm, int wn, int lane, int tid) const {
      const int r = lane & 15, q = lane >> 4;
      const int c0 = n0 + wn * G::WN + 4 * q;
      const int row0 = m0 + wm * G::WM + r;
      float2 *part = e.part + (int64_t)((n0 - g.n_base) / G::BN * G::WGN + wn) * g.M;
      int64_t target[W::TM];
#pragma unroll
      for (int i = 0; i < W::TM; ++i) target[i] = e.target[row0 + 16 * i < g.M ? row0 + 16 * i : g.M - 1];
      const bool edge = n0 + G::BN > g.N;
#pragma unroll
      for (int i = 0; i < W::TM; ++i) {
        const int row = row0 + 16 * i;
        const bool in = row < g.M;
        const RowLogits<G, W> z(w, i, edge, c0, g.N);
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < W::TN; ++j) {
          top = max3(top, z.v[j][0], z.v[j][1]);  // a NaN shows in the sum
          top = max3(top, z.v[j][2], z.v[j][3]);
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float off = top == -INFINITY ? 0.0f : top * kLog2e;  // no finite logit here: the sum is zero, not 0/0
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < W::TN; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) sum += exp_from(z.v[j][x], off);
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (in && q == 0) part[row] = make_float2(top, sum);
        const int64_t t = target[i] - c0;  // column within the lane's blocks
        const bool mine = in && t >= 0 && t < G::WN && (t & 15) < 4;
        if (__any(mine)) {
          float at = 0.0f;
#pragma unroll
          for (int j = 0; j < W::TN; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (t == 16 * j + x) at = z.v[j][x];
          if (mine) e.at[row] = at;
        }
      }
    }
  };
};

// The loss's derivative by a tile of logits, dz = s (e^(z - lse) - [v = t])
// with s = kDzUnit dloss / *top (0 for an ignored row, NaN for a target
// outside the vocabulary whose dloss is not 0), rounded to T; the products after it multiply by
// *top / kDzUnit again.  *top is the largest |dloss|: with the usual dloss, the
// same for all rows, s is a power of two and an improbable target's entry,
// close to -s, rounds to next to nothing, where -dloss itself would give
// every row the same rounding error (measured: 3.0e-3 off instead of 1.7e-3
// over the whole gradient in bf16).  Columns from N up to 8 are zeros.
//
// kDzUnit: binary16 ends at 2^-24, and most entries of a large vocabulary are
// far smaller than 1; bf16 has fp32's range.
template <typename T>
constexpr float kDzUnit = std::is_same_v<T, _Float16> ? 16384.0f : 1.0f;

struct SlopeEpi {
  struct Args {
    uint16_t *dz;
    int64_t pz;
    const float *lse, *dloss;
    int dstep;  // 1, or 0 for one dloss shared by all rows
    const int64_t *target;
    const float *top;
    int64_t ignore, v0, V;  // the piece's first vocabulary row; the whole vocabulary
  };
  template <typename T, class G, class W>
  struct Run {
    __device__ __forceinline__ void operator()(W &w, const Args &e, const FusedProduct &g, char *smem, int m0, int n0,
                                               int wm, int wn, int lane, int tid) const {
      const int r = lane & 15, q = lane >> 4;
      const int c0 = n0 + wn * G::WN + 4 * q;
      const int row0 = m0 + wm * G::WM + r;
      int64_t target[W::TM];
      float lse[W::TM], dloss[W::TM];
#pragma unroll
      for (int i = 0; i < W::TM; ++i) {
        const int row = row0 + 16 * i < g.M ? row0 + 16 * i : g.M - 1;
        target[i] = e.target[row];
        lse[i] = e.lse[row];
        dloss[i] = e.dloss[(int64_t)row * e.dstep];
      }
      const float top = *e.top;
      const bool edge = n0 + G::BN > g.N;
#pragma unroll
      for (int i = 0; i < W::TM; ++i) {
        const int64_t t = target[i];
        const float s = t == e.ignore || dloss[i] == 0.0f ? 0.0f : (t < 0 || t >= e.V) ? NAN : dloss[i] / top * kDzUnit<T>;
        const uint32_t keep = s == 0.0f ? 0u : ~0u;  // an ignored row is zero whatever its logits are
        const float off = lse[i] * kLog2e;
        RowLogits<G, W> z(w, i, edge, c0, g.N);
#pragma unroll
        for (int j = 0; j < W::TN; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) z.v[j][x] = exp_from(z.v[j][x], off);
        const int64_t d = t - e.v0 - c0;  // column within the lane's blocks
        if (__any(d >= 0 && d < G::WN && (d & 15) < 4)) {
#pragma unroll
          for (int j = 0; j < W::TN; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (d == 16 * j + x) z.v[j][x] -= 1.0f;
        }
#pragma unroll
        for (int j = 0; j < W::TN; ++j) {
          const f32x4 v = z.v[j];
          u32x2 p = Mfma<T>::pack4(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
          p[0] &= keep;
          p[1] &= keep;
          char *dst = smem + (wm * G::WM + 16 * i + r) * Staging<G::BN>::PITCH + (wn * G::WN + 16 * j + 4 * q) * 2;
          *reinterpret_cast<u32x2 *>(dst) = p;
        }
      }
      __syncthreads();
      store_tile<G::BM, G::BN, G::THREADS>(smem, Staging<G::BN>::PITCH, 0, e.dz, e.pz, g.M, (g.N + 7) / 8 * 8, m0, n0,
                                           tid);
    }
  };
};

}  // namespace pgemm
