// Host interface of the fused operators between the C ABI (fused_api.hip),
// which checks and plans every call, and the instance units (fused_*.hip),
// one per operator and element type, which launch it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "pgemm.h"

namespace pgemm {

inline int64_t up_to(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
inline int64_t per(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Parts of a call's workspace, each on 256 bytes.
struct Carver {
  int64_t bytes = 0;
  int64_t take(int64_t n) {
    const int64_t at = bytes;
    bytes += up_to(n, 256);
    return at;
  }
};

// 256 x 256 tiles when they alone nearly fill the 256 CUs, else 128 x 128
// (the same rule as the NT calls).
inline bool large_tile(int64_t M, int64_t N, bool dual) { return per(M, 256) * per(N, dual ? 128 : 256) >= 192; }

// Rows up to which the gated block's forward call runs as a product of few
// rows (skinny.hpp) instead of tiles.
constexpr int64_t kSkinnyRows = 64;

// Operands whose rows do not start on 16 bytes are copied into rows that do.
struct GatedPlan {
  bool skinny, padded;
  int64_t d8;        // row pitch of x and W in the products
  int64_t py;        // row pitch of dy
  int64_t x, w, dy;  // workspace offsets
  int64_t bytes;
};

inline GatedPlan plan_gated(int64_t M, int64_t F, int64_t D, bool backward, bool keep) {
  GatedPlan p{};
  Carver c;
  p.skinny = !backward && !keep && M <= kSkinnyRows;
  p.d8 = up_to(D, 8);
  p.py = up_to(2 * F, 8);
  p.padded = !p.skinny && D % 8 != 0;
  if (p.padded) {
    p.x = c.take(M * p.d8 * 2);
    p.w = c.take(2 * F * p.d8 * 2);
  }
  if (backward) p.dy = c.take(M * p.py * 2);
  p.bytes = c.bytes;
  return p;
}

// The derivative by the logits is made and used in pieces of the vocabulary
// of at most this many bytes.
constexpr int64_t kPieceBytes = (int64_t)512 << 20;

struct XentPlan {
  bool padded;
  int64_t d8;
  int64_t parts;  // softmax statistics per row
  int64_t piece;  // vocabulary rows per piece
  int64_t pz;     // row pitch of a piece of dz
  int64_t ps;     // row pitch of the running sum of dx
  int64_t x, w, part, at, dz, sum, scale;
  int64_t bytes;
};

inline XentPlan plan_xent(int64_t M, int64_t V, int64_t D, bool backward) {
  XentPlan p{};
  Carver c;
  p.d8 = up_to(D, 8);
  p.padded = D % 8 != 0;
  if (p.padded) {
    p.x = c.take(M * p.d8 * 2);
    p.w = c.take(V * p.d8 * 2);
  }
  if (!backward) {
    // wave columns: 128 on the large tile, 32 on the small one
    p.parts = large_tile(M, V, false) ? per(V, 256) * 2 : per(V, 128) * 4;
    p.part = c.take(p.parts * M * 8);
    p.at = c.take(M * 4);
  } else {
    p.piece = kPieceBytes / (2 * (M > 0 ? M : 1)) / 256 * 256;
    if (p.piece < 256) p.piece = 256;
    if (p.piece > V) p.piece = V;
    p.pz = up_to(p.piece, 8);
    p.ps = up_to(D, 4);
    p.dz = c.take(M * p.pz * 2);
    if (p.piece < V) p.sum = c.take(M * p.ps * 4);
    p.scale = c.take(8);
  }
  p.bytes = c.bytes;
  return p;
}

struct GatedCall {
  const uint16_t *x, *w, *dh;
  const float *saved_in;
  uint16_t *h, *dx, *dw;
  float *saved;
  int64_t M, F, D;
  int act;
  char *ws;
  hipStream_t stream;
  int dev;
};

struct XentCall {
  const uint16_t *x, *w;
  const int64_t *target;
  const float *dloss, *lse_in;
  int dstep;
  float *loss, *lse;
  uint16_t *dx, *dw;
  int64_t M, V, D, ignore;
  char *ws;
  hipStream_t stream;
  int dev;
};

struct Q4Call {
  const uint16_t *x;
  const uint8_t *q;
  const uint16_t *scale;
  const uint8_t *zero;
  uint16_t *out;
  int64_t M, N, K;
  int group;
  bool gated;
  int act;
  hipStream_t stream;
  int dev;
};

pgemm_status gated_f16(const GatedCall &);
pgemm_status gated_bf16(const GatedCall &);
pgemm_status gated_bwd_f16(const GatedCall &);
pgemm_status gated_bwd_bf16(const GatedCall &);
pgemm_status xent_f16(const XentCall &);
pgemm_status xent_bf16(const XentCall &);
pgemm_status xent_bwd_f16(const XentCall &);
pgemm_status xent_bwd_bf16(const XentCall &);
pgemm_status q4_f16(const Q4Call &);
pgemm_status q4_bf16(const Q4Call &);

// From pgemm_api.hip: the current device if it is a gfx950, and the workspace
// registered for (device, stream), with the registry locked until the
// caller's kernels are enqueued.
pgemm_status checked_device(int *dev);
pgemm_status stream_workspace(int dev, void *stream, int64_t bytes, std::unique_lock<std::mutex> *lock, char **ws);

}  // namespace pgemm
