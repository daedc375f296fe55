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

// How a tiled product is cut: output tiles of 256 x 256 or 128 x 128, and
// pieces of K whose fp32 partial sums a second kernel adds up in order.  Small
// tiles that are at most one to a CU run with four ring slots (`deep`): alone
// on a CU a tile waits for its loads most of the time, and with two slots it
// took 0.72 us a K tile.
//
// The cut that takes least by these times, in microseconds, which the kernels
// were measured to need for the tiles of one CU (K tiles of 64):
//   large, one to a CU:         1.5 a K tile and 12 to fill and store
//   small, deep, one to a CU:   0.45 and 6
//   small, two to a CU:         1.0 and 9 (0.72 and 7 for one left over)
// with K along the rows of both operands.  With K down the rows of one, 256 deep
// tiles take 0.60 a K tile in 86 of them and 0.63 to 0.73 in 196, which the cut
// does not go by: such long products may be better off in pieces of large tiles.
// By these, a large tile has the work of four small ones for less than the time of
// four, but leaves CUs idle when there are fewer than 256, or few more than a
// multiple.  Pieces cost a second launch (4) and their sums' way to memory and
// back (4 MB a microsecond).  Examples: 2048 x 2048 x 4096 takes 39 us in 256
// small deep tiles, 52 with two slots; 8192 x 2048 x 2048 takes 58 in 256 large
// ones and 80 in 1024 small ones.
//
// Large tiles that do not come out at whole rounds of 256 may leave the rest to
// small ones in a launch of its own (`cut_m` rows or `cut_n` columns by large
// tiles): 784 tiles take three rounds and a quarter's time instead of four.
struct Tiling {
  bool large, deep;
  int split;
  int64_t k_chunk;       // a multiple of 64 when split
  int64_t cut_m, cut_n;  // 0: one launch
  double us;             // what the cut was taken for
};

constexpr int kMaxPieces = 16;
constexpr int64_t kMaxWorkItems = (int64_t)1 << 32;  // a dispatch's are fewer

inline double small_tiles_us(int64_t blocks, double steps) {
  if (blocks <= 256) return 0.45 * steps + 6.0;
  const int64_t rest = blocks % 512;
  return (double)(blocks / 512 + (rest > 256)) * (steps + 9.0) + (rest > 0 && rest <= 256 ? 0.72 * steps + 7.0 : 0.0);
}
inline double large_tiles_us(int64_t blocks, double steps) { return (double)per(blocks, 256) * (1.5 * steps + 12.0); }

// How a product may be cut: in pieces of K, and by rows (a kernel whose results
// depend on the width of a tile needs the same one in all rows).
struct Cuts {
  bool k, m;
};

inline Tiling plan_tiles(int64_t M, int64_t N, int64_t K, bool dual, Cuts may) {
  Tiling best{false, false, 1, K, 0, 0, 0.0};
  double least = -1.0;
  auto take = [&](double us, const Tiling &t) {
    if (least >= 0.0 && us >= least) return;
    least = us;
    best = t;
    best.us = us;
  };
  for (int large = 0; large < 2; ++large) {
    const int64_t t = large ? 256 : 128;
    const int64_t tiles = per(M, t) * per(N, dual ? t / 2 : t);
    for (int want = 1; want <= (may.k ? kMaxPieces : 1); ++want) {
      const int64_t chunk = want == 1 ? K : up_to(per(K, want), 64);
      const int split = chunk > 0 ? (int)per(K, chunk) : 1;
      if (split != want || (want > 1 && chunk < 256)) continue;
      const double steps = (double)per(chunk, 64);
      const int64_t blocks = tiles * split;
      if (blocks * (large ? 256 : 512) >= kMaxWorkItems) continue;
      double us = large ? large_tiles_us(blocks, steps) : small_tiles_us(blocks, steps);
      if (split > 1) us += 4.0 + (double)M * (double)N * (8.0 * split + 2.0) / 4e6;
      take(us, Tiling{large != 0, !large && blocks <= 256, split, chunk, 0, 0, 0.0});
    }
  }
  const double steps = (double)per(K, 64);
  const int64_t tm = per(M, 256), bn = dual ? 128 : 256, tn = per(N, bn), rounds = tm * tn / 256;
  if (rounds > 0) {
    auto fits = [](int64_t rest) { return rest * 512 < kMaxWorkItems; };
    const int64_t n = rounds * 256 / tm, m = may.m ? rounds * 256 / tn : 0;
    if (n > 0 && n < tn) {
      const int64_t rest = per(M, 128) * per(N - n * bn, bn / 2);
      if (fits(rest))
        take(large_tiles_us(tm * n, steps) + 3.0 + small_tiles_us(rest, steps), Tiling{true, rest <= 256, 1, K, 0, n * bn, 0.0});
    }
    if (m > 0 && m < tm) {
      const int64_t rest = per(M - m * 256, 128) * per(N, bn / 2);
      if (fits(rest))
        take(large_tiles_us(m * tn, steps) + 3.0 + small_tiles_us(rest, steps), Tiling{true, rest <= 256, 1, K, m * 256, 0, 0.0});
    }
  }
  return best;
}

// The same cut for a product with fewer rows, columns or less K.
inline Tiling shortened(Tiling t, int64_t K) {
  if (t.split > 1) {
    t.split = (int)per(K, t.k_chunk);
    if (t.split < 1) t.split = 1;
  }
  if (t.split == 1) t.k_chunk = K;
  t.cut_m = t.cut_n = 0;
  return t;
}

// Bytes of a product's partial sums (rows of a multiple of 4).
inline int64_t piece_bytes(const Tiling &t, int64_t M, int64_t N) {
  return t.split > 1 ? t.split * M * up_to(N, 4) * 4 : 0;
}

// The gated block's forward call as a product of few rows (skinny.hpp), up to
// 256 of them: microseconds, by what its workgroups of 16 hidden columns were
// measured to take for a block of 128 k of up to 32 or 64 tokens.  Rows that do
// not start on 16 bytes load slower there, but need no padded copy.  100 x 800 x
// 4096 takes 14 us so and 25 in tiles, 64 x 12288 x 4096 47 and 32.
constexpr int64_t kSkinnyRows = 256;
inline double few_rows_us(int64_t M, int64_t F, int64_t D) {
  const int64_t blocks = per(D, 128), groups = per(F, 16) * per(M, M <= 16 ? 16 : M <= 32 ? 32 : 64);
  const int64_t per_cu = groups > 256 ? per(groups * blocks, 256) : blocks;
  return 3.5 + (M <= 32 ? 0.28 : 0.45) * (D % 8 ? 1.8 : 1.0) * (double)per_cu;
}

// Operands whose rows do not start on 16 bytes are copied into rows that do.
struct GatedPlan {
  bool skinny, padded;
  int64_t d8;        // row pitch of x and W in the products
  int64_t py;        // row pitch of dy
  int64_t x, w, dy, part;  // workspace offsets
  Tiling forward, dx, dw;
  int64_t bytes;
};

inline GatedPlan plan_gated(int64_t M, int64_t F, int64_t D, bool backward, bool keep) {
  GatedPlan p{};
  Carver c;
  p.d8 = up_to(D, 8);
  p.py = up_to(2 * F, 8);
  p.forward = plan_tiles(M, F, p.d8, true, Cuts{false, true});
  if (!backward && !keep && M <= kSkinnyRows) {
    const double copies = D % 8 ? 3.0 + (double)(M + 2 * F) * (double)D / 1.1e6 : 0.0;  // 4.4 MB a microsecond
    p.skinny = few_rows_us(M, F, D) < p.forward.us + copies;
  }
  p.padded = !p.skinny && D % 8 != 0;
  if (p.padded) {
    p.x = c.take(M * p.d8 * 2);
    p.w = c.take(2 * F * p.d8 * 2);
  }
  if (backward) {
    p.dy = c.take(M * p.py * 2);
    p.dx = plan_tiles(M, D, 2 * F, false, Cuts{true, true});
    p.dw = plan_tiles(2 * F, D, M, false, Cuts{true, true});
    const int64_t a = piece_bytes(p.dx, M, D), b = piece_bytes(p.dw, 2 * F, D);
    p.part = c.take(a > b ? a : b);
  }
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
  int64_t piece;  // vocabulary rows per piece, the last one's may be fewer
  int64_t pz;     // row pitch of a piece of dz
  int64_t ps;     // row pitch of the running sum of dx
  int64_t x, w, part, at, dz, sum, scale;
  Tiling logits, dx, dw;  // of a whole piece
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
    p.logits = plan_tiles(M, V, p.d8, false, Cuts{false, false});
    // wave columns: 128 on the large tile, 32 on the small one
    const int64_t wide = !p.logits.large ? 0 : p.logits.cut_n ? p.logits.cut_n : V;
    p.parts = per(wide, 256) * 2 + (wide < V ? per(V - wide, 128) * 4 : 0);
    p.part = c.take(p.parts * M * 8);
    p.at = c.take(M * 4);
  } else {
    p.piece = kPieceBytes / (2 * (M > 0 ? M : 1)) / 256 * 256;
    if (p.piece < 256) p.piece = 256;
    // pieces alike, so that the last one is no short one
    if (p.piece < V)
      p.piece = up_to(per(V, per(V, p.piece)), 256);
    else
      p.piece = V;
    p.pz = up_to(p.piece, 8);
    p.ps = up_to(D, 4);
    p.logits = plan_tiles(M, p.piece, p.d8, false, Cuts{false, true});
    p.dx = plan_tiles(M, D, p.piece, false, Cuts{true, true});
    p.dw = plan_tiles(p.piece, D, M, false, Cuts{true, true});
    const int64_t a = piece_bytes(p.dx, M, D), b = piece_bytes(p.dw, p.piece, D);
    p.part = c.take(a > b ? a : b);
    p.dz = c.take(M * p.pz * 2);
    if (p.piece < V) p.sum = c.take(M * p.ps * 4);
    p.scale = c.take(8);
  }
  p.bytes = c.bytes;
  return p;
}

// Workgroups of 1024 that join the softmax statistics, 16 rows each at a time:
// all of them up to 2^24 rows, which then take several.
inline int64_t join_groups(int64_t M) { return per(M, 16) < (1 << 20) ? per(M, 16) : 1 << 20; }

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
