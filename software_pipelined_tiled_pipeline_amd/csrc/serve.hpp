// Host interface of the serving operators (8-bit products, mixture of experts,
// choice of a token) between the C ABI (serve_api.hip), which checks and plans
// every call, and the instance units (serve_*.hip).
#pragma once

#include "fused.hpp"

namespace pgemm {

// The largest K whose sums of products of two 8-bit integers stay in int32.
constexpr int64_t kI8MaxK = ((int64_t)1 << 17) - 16;

// How an 8-bit product runs: by few_rows kernels up to 64 tokens, else in tiles.
constexpr int64_t kI8FewRows = 64;

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
  p.few = M <= kI8FewRows;
  p.own = p.few && !quantized && M <= 4 && K >= 8 && K <= 8192;
  if (!quantized && !p.own) {
    p.q = c.take(M * width);
    p.s = c.take(M * 4);
  }
  if (!p.few) {
    p.tiles = plan_tiles(M, N, width / 2, gated, Cuts{!gated, true});
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
constexpr int64_t kMoeChunkTokens = 64, kMoeMaxExperts = 1024, kMoeMaxTop = 32, kMoeMaxTokens = 32768, kMoeMaxSplits = 8;
constexpr int64_t kMoeDownColumns = 32;  // of a workgroup of the second products
// hidden values, so that those of a chunk's choices stay below 2^31 bytes
constexpr int64_t kMoeMaxHidden = (int64_t)1 << 17;

struct MoePlan {
  int64_t slots;    // experts a chunk may reach, or, if fewer, its choices
  bool by_choice;
  int64_t splits;   // workgroups that share 32 columns of y
  int64_t groups;   // such columns of all chunks
  int64_t logits, experts, weights, h, tops, counts, lists, partial, arrived;  // workspace offsets
  int64_t bytes;
};

inline MoePlan plan_moe(int64_t M, int64_t E, int64_t D, int64_t F, int64_t top_k) {
  MoePlan p{};
  Carver c;
  const int64_t chunks = per(M, kMoeChunkTokens), most = (M < kMoeChunkTokens ? M : kMoeChunkTokens) * top_k;
  p.by_choice = most < E;
  p.slots = p.by_choice ? most : E;
  // The second products run in as many workgroups as give each CU two, but none with less than two blocks of K a wave
  // (eight of them) where every choice is of another expert.
  p.groups = per(D, kMoeDownColumns) * chunks;
  const int64_t blocks = (M * top_k < E ? M * top_k : E) * per(F, 128);
  p.splits = p.groups > 0 ? 512 / p.groups : 1;
  if (p.splits > blocks / 16) p.splits = blocks / 16;
  p.splits = p.splits < 1 ? 1 : p.splits > kMoeMaxSplits ? kMoeMaxSplits : p.splits;
  p.logits = c.take(M * E * 8);
  p.experts = c.take(M * top_k * 4);
  p.weights = c.take(M * top_k * 4);
  p.h = c.take(M * top_k * F * 4);
  p.tops = c.take(M * top_k * 4);
  p.counts = c.take(chunks * p.slots * 4);
  p.lists = c.take(chunks * p.slots * kMoeChunkTokens * 2);
  p.arrived = c.take(p.groups * 4);
  if (p.splits > 1) p.partial = c.take(p.splits * M * D * 4);
  p.bytes = c.bytes;
  return p;
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
