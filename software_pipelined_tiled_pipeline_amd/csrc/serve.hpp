// Host interface of the serving operators (8-bit products, mixture of experts,
// choice of a token) between the C ABI (serve_api.hip), which checks and plans
// every call, and the instance units (serve_*.hip).
#pragma once

#include "fused.hpp"

namespace pgemm {

// The largest K whose sums of products of two 8-bit integers stay in int32.
constexpr int64_t kI8MaxK = ((int64_t)1 << 17) - 16;

// An 8-bit product of up to 256 tokens by the kernel for few of them, or in
// tiles, whichever is expected to take less: microseconds, by what a workgroup's 256
// bytes of K were measured to take with 16, 32 or 64 tokens, where at least half of
// the CUs have one, and by plan_tiles (whose times are those of 16-bit products of as
// many bytes), or the weights' way from memory where that is longer.  The first is
// off by a fifth where the last round of workgroups is a short one: of the sizes here
// it takes 64 x 12288 x 4096 and 64 x 8192 x 8192 the slower way.
// Measured, tiles and few tokens, for tokens x columns x K:
//   8 x 4096 x 4096   10.1  6.8     64 x 12288 x 4096  20.5 22.5     128 x 4096 x 4096   15.7 10.4
//   8 x 8192 x 8192   17.5 14.1     64 x 8192 x 8192   25.1 21.1     128 x 8192 x 8192   29.8 36.9
//   8 x 28672 x 4096  29.4 23.1     64 x 28672 x 4096  30.4 40.0     128 x 28672 x 4096  31.9 64.4
// and gated
//   32 x 12288 x 4096  26.9 22.1    64 x 12288 x 4096  27.5 33.0     64 x 1024 x 8192    25.8 15.0
constexpr int64_t kI8FewRows = 256;
inline double i8_few_us(int64_t M, int64_t groups, int64_t width) {
  const double mine = M <= 16 ? 0.36 : M <= 32 ? 0.42 : 0.6;
  return 3.5 + mine * (double)per(width, 256) * (groups > 128 ? (double)groups : 128.0) / 256.0;
}
inline double i8_tiles_us(const Tiling &t, int64_t rows, int64_t width) {
  const double bytes = 4.0 + (double)rows * (double)width / 4.6e6;
  return t.us > bytes ? t.us : bytes;
}

struct I8Plan {
  bool few;
  bool own;         // few tokens of 16 bits: each workgroup makes them integers
  int64_t q, s;     // workspace offsets of the tokens' integers and scales,
  int64_t part;     // and of the sums of pieces of K
  Tiling tiles;
  int64_t bytes;
};

inline I8Plan plan_i8(int64_t M, int64_t N, int64_t K, bool gated, bool quantized) {
  I8Plan p{};
  Carver c;
  const int64_t width = up_to(K, 16);
  p.tiles = plan_tiles(M, N, width / 2, gated, Cuts{!gated, true});
  const int64_t groups = per(N, gated ? 16 : 32) * per(M, M <= 16 ? 16 : M <= 32 ? 32 : 64);
  p.few = M <= kI8FewRows && i8_few_us(M, groups, width) < i8_tiles_us(p.tiles, gated ? 2 * N : N, width);
  p.own = p.few && !quantized && M <= 4 && K >= 8 && K <= 8192;
  if (!quantized && !p.own) {
    p.q = c.take(M * width);
    p.s = c.take(M * 4);
  }
  if (!p.few) {
    p.part = c.take(piece_bytes(p.tiles, M, N));
  }
  p.bytes = c.bytes;
  return p;
}

struct QuantCall {
  const uint16_t *x;
  int8_t *q;
  float *scale;
  int64_t M, K;
  hipStream_t stream;
};

struct I8Call {
  const uint16_t *x;  // tokens of 16 bits, or null:
  const int8_t *q;    // integers and scales
  const float *xs;
  const int8_t *w;
  const float *ws;
  uint16_t *out;
  int64_t M, N, K;
  bool gated;
  int act;
  char *workspace;
  hipStream_t stream;
  int dev;
};

// The mixture of experts takes tokens in chunks.
constexpr int64_t kMoeChunkTokens = 64, kMoeMaxExperts = 1024, kMoeMaxTop = 32, kMoeMaxTokens = 32768;
// hidden values, so that those of a chunk's choices stay below 2^31 bytes
constexpr int64_t kMoeMaxHidden = (int64_t)1 << 17;

struct MoePlan {
  int64_t slots;    // experts a chunk may reach, or, if fewer, its choices
  bool by_choice;
  int64_t logits, experts, weights, h, tops, products;  // workspace offsets
  int64_t bytes;
};

inline MoePlan plan_moe(int64_t M, int64_t E, int64_t D, int64_t F, int64_t top_k) {
  MoePlan p{};
  Carver c;
  const int64_t most = (M < kMoeChunkTokens ? M : kMoeChunkTokens) * top_k;
  p.by_choice = most < E;
  p.slots = p.by_choice ? most : E;
  p.logits = c.take(M * E * 8);
  p.experts = c.take(M * top_k * 4);
  p.weights = c.take(M * top_k * 4);
  p.h = c.take(M * top_k * F * 4);
  p.tops = c.take(M * top_k * 4);
  if (top_k > 1) p.products = c.take(M * top_k * D * 4);
  p.bytes = c.bytes;
  return p;
}

// Blocks of 16 rows (second products: two rows a token) that a workgroup takes at a
// time, by how many an expert has on average; waves along K so that all workgroups
// together give each CU about sixteen.  Second products, the whole layer's time: 64
// tokens' two of 8 experts of 4096 x 1280 in bf16 75 us in four blocks, 77 in two;
// their eight of 64 404 us in f16 in two blocks, 412 in one.
struct MoeCut {
  int blocks, waves;
};

inline MoeCut moe_cut(int64_t M, int64_t E, int64_t D, int64_t F, int64_t top_k, bool down) {
  const int64_t mean = (M < kMoeChunkTokens ? M : kMoeChunkTokens) * top_k * (down ? 2 : 1) / E;
  const int64_t groups = (down ? per(D, 32) : per(F, 16)) * plan_moe(M, E, D, F, top_k).slots * per(M, kMoeChunkTokens);
  return MoeCut{mean > 24 ? 4 : mean > 8 ? 2 : 1, mean > 24 || groups > 512 ? 4 : 8};
}

struct MoeCall {
  const uint16_t *x, *router, *w, *down;
  uint16_t *y;
  int32_t *experts;  // null: in the workspace
  float *weights;
  int64_t M, E, D, F, top_k;
  bool normalize;
  int act;
  char *workspace;
  hipStream_t stream;
  int dev;
};

struct SampleCall {
  const uint16_t *logits;
  const float *u, *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p;
  int shared;  // pgemm_sample_setting bits: one value for all rows
  int64_t *token;
  int64_t M, V;
  hipStream_t stream;
  int dev;
};

pgemm_status moe_f16(const MoeCall &);
pgemm_status moe_bf16(const MoeCall &);
pgemm_status sample_f16(const SampleCall &);
pgemm_status sample_bf16(const SampleCall &);
pgemm_status quant_i8_f16(const QuantCall &);
pgemm_status quant_i8_bf16(const QuantCall &);
pgemm_status i8_f16(const I8Call &);
pgemm_status i8_bf16(const I8Call &);

}  // namespace pgemm
