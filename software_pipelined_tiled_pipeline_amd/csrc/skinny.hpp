// The gated block act(x Wg^T) * (x Wu^T) for few rows (tokens) and 16-bit weights,
// bound by reading the weights once.
//
// A workgroup owns 16 gate rows, the same 16 up rows and all of K; its waves take
// blocks of 128 k in turn, so that a weight row's loads are in flight on
// several waves at once, and add their sums up in LDS at the end.  Weights are
// not staged in LDS: four lanes load 64 bytes of a row, so that a load is 16
// requests and not one a lane, the values change lanes to where
// v_mfma_f32_16x16x32 wants them, row l % 16, and meet the tokens (16 of
// them, those past M repeat the last one) as the other operand:
//   lane l, register r of an accumulator: token 4 (l / 16) + r, weight row l % 16.
//
// One token at 4096 x 12288 gated takes 34.6 us, 5.8 TB/s, also where no cache
// holds the weights.  With one row a lane, each a request of its own, 18 tokens at
// 421 x 3264 took 12.7 us, 7.4 in whole lines.  More tokens read x again for every 32 weight
// rows, and from about 64 on tiles take less (few_rows_us).
#pragma once

#include "few_rows.hpp"

namespace pgemm {

struct SkinnyArgs {
  const uint16_t *x;  // [M][K]
  const uint16_t *w;  // [2 N][K]
  uint16_t *out;      // [M][N]
  int M, N, K;
  int act;
};

// The 16 bytes of lane 4 (l % 16) + l / 16, for lane l.
__device__ __forceinline__ u32x4 to_rows(u32x4 v, int from) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v[i]);
  return r;
}

// A wave's K loop.  Whole blocks of 128 k (four MFMA steps) are loaded a block
// ahead of their use, without bounds checks: a token past M repeats the last
// one, a weight row past the end too (neither reaches a stored value), and a
// block that K ends in is left to one wave's guarded loads after the loop.
// Addresses are a base that is the same for the wave and moves along K, and a
// lane's offset of 32 bits.
template <typename T, int MT>
struct SkinnyRun {
  using F = Frag8<T>;
  static constexpr int NT = 2;                // blocks of weight rows: gate, up
  static constexpr int XD = MT == 1 ? 4 : 2;  // steps that x is loaded ahead

  const SkinnyArgs &a;
  const char *xbase[MT], *wbase[NT];  // of the wave's blocks of 16 rows
  uint32_t xoff[MT], woff[NT];        // what this lane loads there: row l / 4, 16-byte piece l % 4
  int from;                           // the lane its fragments come from, in bytes
  f32x4 tot[MT][NT];
  u32x4 xr[XD][MT], wr[4][NT];  // the next steps' fragments

  __device__ __forceinline__ SkinnyRun(const SkinnyArgs &args) : a(args) {}

  // Rows of a block of 16 from row0 on: the offset of its row r, the last one's past the end.
  __device__ __forceinline__ static uint32_t row_offset(int row0, int r, int rows, uint32_t pitch) {
    return (uint32_t)((row0 + r < rows ? row0 + r : rows - 1) - (row0 < rows ? row0 : rows - 1)) * pitch;
  }

  __device__ __forceinline__ void init(int lane, int m0, int n0) {
    const uint32_t pitch = (uint32_t)a.K * 2u;
    from = (4 * (lane & 15) + (lane >> 4)) * 4;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row0 = m0 + 16 * m;
      xbase[m] = reinterpret_cast<const char *>(a.x) + (int64_t)(row0 < a.M ? row0 : a.M - 1) * pitch;
      xoff[m] = row_offset(row0, lane >> 2, a.M, pitch) + 16u * (lane & 3);
    }
#pragma unroll
    for (int b = 0; b < NT; ++b) {
      wbase[b] = reinterpret_cast<const char *>(a.w) + ((n0 < a.N ? n0 : a.N - 1) + (int64_t)b * a.N) * pitch;
      woff[b] = row_offset(n0, lane >> 2, a.N, pitch) + 16u * (lane & 3);
    }
  }

  __device__ __forceinline__ void load_x(int slot, int k) {
#pragma unroll
    for (int m = 0; m < MT; ++m) xr[slot][m] = load_at<u32x4_any>(xbase[m] + (int64_t)k * 2, xoff[m]);
  }
  __device__ __forceinline__ void load_w(int s, int kb) {
#pragma unroll
    for (int b = 0; b < NT; ++b) wr[s][b] = load_at<u32x4_any>(wbase[b] + (int64_t)kb * 256 + s * 64, woff[b]);
  }

  // Block kb, while block nk loads.
  template <bool MORE>
  __device__ __forceinline__ void whole(int kb, int nk) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 x[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) x[m] = to_rows(xr[s % XD][m], from);
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const u32x4 w = to_rows(wr[s][b], from);
#pragma unroll
        for (int m = 0; m < MT; ++m) tot[m][b] = F::mma(x[m], w, tot[m][b]);
      }
      if (MORE) load_w(s, nk);
      // the slot of step s takes step s + XD
      if (s + XD < 4)
        load_x(s % XD, kb * 128 + 32 * (s + XD));
      else if (MORE)
        load_x(s % XD, nk * 128 + 32 * (s + XD - 4));
    }
  }

  // Places first, first + step, .. below `full` in the order of blocks that
  // starts at `turn`, and the block that K ends in if it is `tail`.
  __device__ __forceinline__ void run(int lane, int m0, int n0, int first, int step, int full, int turn, bool tail) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int b = 0; b < NT; ++b) tot[m][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (first < full) {
      auto block = [&](int place) { return place + turn < full ? place + turn : place + turn - full; };
      int at = first, kb = block(at);
#pragma unroll
      for (int s = 0; s < 4; ++s) load_w(s, kb);
#pragma unroll
      for (int s = 0; s < XD; ++s) load_x(s, kb * 128 + 32 * s);
      for (at += step; at < full; at += step) {
        const int nk = block(at);
        whole<true>(kb, nk);
        kb = nk;
      }
      whole<false>(kb, kb);
    }
    if (!tail) return;
    // a lane loads its own fragments
    const int c = lane & 15, q = lane >> 4;
    const uint32_t pitch = (uint32_t)a.K * 2u;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = full * 128 + 32 * s + 8 * q;
      u32x4 x[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        x[m] = load_tail(reinterpret_cast<const uint16_t *>(xbase[m] + row_offset(m0 + 16 * m, c, a.M, pitch)), k, a.K);
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const u32x4 f = load_tail(reinterpret_cast<const uint16_t *>(wbase[b] + row_offset(n0, c, a.N, pitch)), k, a.K);
#pragma unroll
        for (int m = 0; m < MT; ++m) tot[m][b] = F::mma(x[m], f, tot[m][b]);
      }
    }
  }
};

template <typename T, int MT, int WAVES>
__global__ void __launch_bounds__(WAVES * 64) skinny_kernel(SkinnyArgs a) {
  constexpr int NT = SkinnyRun<T, MT>::NT;
  extern __shared__ __attribute__((aligned(16))) float sums[];  // [WAVES][MT * NT * 4][64]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * MT * 16;

  SkinnyRun<T, MT> job(a);
  job.init(lane, m0, n0);
  const int full = a.K / 128;
  // Each workgroup starts at another block: rows are often a multiple of the
  // memory channels' interleave apart, and all would meet on the same few.
  const int turn = full > 0 ? (int)((blockIdx.x * 0x9E3779B1u >> 12) % (unsigned)full) : 0;
  job.run(lane, m0, n0, wave, WAVES, full, turn, a.K % 128 != 0 && wave == full % WAVES);
  constexpr int VALS = MT * NT * 4;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[(wave * VALS + (m * NT + b) * 4 + r) * 64 + lane] = job.tot[m][b][r];
  __syncthreads();
  join_and_store<T, true, MT, NT>(sums, WAVES, VALS * 64, wave, WAVES, lane, a.act, a.out, a.M, a.N, m0, n0,
                                  [](float v, int, int64_t) { return v; });
}

}  // namespace pgemm
