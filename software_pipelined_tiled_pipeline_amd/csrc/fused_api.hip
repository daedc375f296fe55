// C ABI of the fused operators: argument checks, workspaces, dispatch by type.
//
// Arguments are checked before any HIP call, and nothing is enqueued for a
// call that is refused.
#include "api_checks.hpp"

namespace {

using namespace pgemm;
using namespace pgemm::api;

pgemm_status check_gated(int64_t M, int64_t F, int64_t D, int act) {
  if (!dim(M) || !pitch(F < 0 ? F : 2 * F) || !pitch(D) || !act_ok(act)) return PGEMM_ERR_SHAPE;
  if (!grid_fits(M, F) || !grid_fits(M, D) || !grid_fits(2 * F, D)) return PGEMM_ERR_SHAPE;
  return PGEMM_OK;
}

template <typename Launch>
pgemm_status gated(Launch launch, const uint16_t *x, const uint16_t *w, uint16_t *h, float *saved, int64_t M, int64_t F,
                   int64_t D, int act, void *stream) {
  pgemm_status st = check_gated(M, F, D, act);
  if (st != PGEMM_OK) return st;
  if (missing(x, M * D) || missing(w, F * D) || missing(h, M * F)) return PGEMM_ERR_NULL;
  if (off16(x) || off16(w) || off16(h) || off16(saved)) return PGEMM_ERR_ALIGN;
  if (M == 0 || F == 0) return PGEMM_OK;
  Site s;
  st = s.open(stream, plan_gated(M, F, D, false, saved != nullptr).bytes);
  if (st != PGEMM_OK) return st;
  GatedCall c{};
  c.x = x;
  c.w = w;
  c.h = h;
  c.saved = saved;
  c.M = M;
  c.F = F;
  c.D = D;
  c.act = act;
  c.ws = s.ws;
  c.stream = static_cast<hipStream_t>(stream);
  c.dev = s.dev;
  return launch(c);
}

template <typename Launch>
pgemm_status gated_bwd(Launch launch, const uint16_t *dh, const uint16_t *x, const uint16_t *w, const float *saved,
                       uint16_t *dx, uint16_t *dw, int64_t M, int64_t F, int64_t D, int act, void *stream) {
  pgemm_status st = check_gated(M, F, D, act);
  if (st != PGEMM_OK) return st;
  if (missing(dh, M * F) || missing(x, M * D) || missing(w, F * D) || missing(dx, M * D) || missing(dw, F * D))
    return PGEMM_ERR_NULL;
  if (off16(dh) || off16(x) || off16(w) || off16(saved) || off16(dx) || off16(dw)) return PGEMM_ERR_ALIGN;
  if (D == 0 || (M == 0 && F == 0)) return PGEMM_OK;
  Site s;
  st = s.open(stream, plan_gated(M, F, D, true, false).bytes);
  if (st != PGEMM_OK) return st;
  GatedCall c{};
  c.dh = dh;
  c.x = x;
  c.w = w;
  c.saved_in = saved;
  c.dx = dx;
  c.dw = dw;
  c.M = M;
  c.F = F;
  c.D = D;
  c.act = act;
  c.ws = s.ws;
  c.stream = static_cast<hipStream_t>(stream);
  c.dev = s.dev;
  return launch(c);
}

pgemm_status check_xent(int64_t M, int64_t V, int64_t D) {
  if (!dim(M) || !dim(V) || !pitch(D) || (M > 0 && V == 0)) return PGEMM_ERR_SHAPE;
  if (!grid_fits(M, V) || !grid_fits(M, D) || !grid_fits(V, D)) return PGEMM_ERR_SHAPE;
  return PGEMM_OK;
}

template <typename Launch>
pgemm_status xent(Launch launch, const uint16_t *x, const uint16_t *w, const int64_t *target, float *loss, float *lse,
                  int64_t M, int64_t V, int64_t D, int64_t ignore, void *stream) {
  pgemm_status st = check_xent(M, V, D);
  if (st != PGEMM_OK) return st;
  if (missing(x, M * D) || missing(w, V * D) || missing(target, M) || missing(loss, M) || missing(lse, M))
    return PGEMM_ERR_NULL;
  if (off16(x) || off16(w) || off16(target) || off16(loss) || off16(lse)) return PGEMM_ERR_ALIGN;
  if (M == 0) return PGEMM_OK;
  Site s;
  st = s.open(stream, plan_xent(M, V, D, false).bytes);
  if (st != PGEMM_OK) return st;
  XentCall c{};
  c.x = x;
  c.w = w;
  c.target = target;
  c.loss = loss;
  c.lse = lse;
  c.M = M;
  c.V = V;
  c.D = D;
  c.ignore = ignore;
  c.ws = s.ws;
  c.stream = static_cast<hipStream_t>(stream);
  c.dev = s.dev;
  return launch(c);
}

template <typename Launch>
pgemm_status xent_bwd(Launch launch, const float *dloss, int dstep, const uint16_t *x, const uint16_t *w,
                      const int64_t *target, const float *lse, uint16_t *dx, uint16_t *dw, int64_t M, int64_t V,
                      int64_t D, int64_t ignore, void *stream) {
  pgemm_status st = check_xent(M, V, D);
  if (st != PGEMM_OK) return st;
  if (dstep != 0 && dstep != 1) return PGEMM_ERR_SHAPE;
  if (missing(dloss, M) || missing(x, M * D) || missing(w, V * D) || missing(target, M) || missing(lse, M) ||
      missing(dx, M * D) || missing(dw, V * D))
    return PGEMM_ERR_NULL;
  if (off16(x) || off16(w) || off16(target) || off16(lse) || off16(dx) || off16(dw)) return PGEMM_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(dloss) & 3u) != 0) return PGEMM_ERR_ALIGN;
  if (D == 0 || V == 0) return PGEMM_OK;
  Site s;
  st = s.open(stream, plan_xent(M, V, D, true).bytes);
  if (st != PGEMM_OK) return st;
  XentCall c{};
  c.dloss = dloss;
  c.dstep = dstep;
  c.x = x;
  c.w = w;
  c.target = target;
  c.lse_in = lse;
  c.dx = dx;
  c.dw = dw;
  c.M = M;
  c.V = V;
  c.D = D;
  c.ignore = ignore;
  c.ws = s.ws;
  c.stream = static_cast<hipStream_t>(stream);
  c.dev = s.dev;
  return launch(c);
}

template <typename Launch>
pgemm_status q4(Launch launch, const uint16_t *x, const uint8_t *q, const uint16_t *scale, const uint8_t *zero,
                uint16_t *out, int64_t M, int64_t N, int64_t K, int64_t group, bool gated, int act, void *stream) {
  const int64_t rows = gated ? 2 * N : N;
  if (!dim(M) || !dim(N) || !dim(rows) || !pitch(K) || group <= 0 || group % 32 != 0 || group >= (int64_t)1 << 31 || !act_ok(act))
    return PGEMM_ERR_SHAPE;
  // tokens are the grid's second dimension, at least 16 a workgroup
  if (per(M, 16) > 65535 || per(N, 16) * 512 >= kMaxWorkItems) return PGEMM_ERR_SHAPE;
  const int64_t need = K > 0 ? rows : 0;
  if (missing(x, M * K) || missing(q, need) || missing(scale, need) || missing(out, M * N)) return PGEMM_ERR_NULL;
  if (off16(x) || off16(q) || off16(scale) || off16(zero) || off16(out)) return PGEMM_ERR_ALIGN;
  if (M == 0 || N == 0) return PGEMM_OK;
  Site s;
  pgemm_status st = s.open(stream, 0);
  if (st != PGEMM_OK) return st;
  Q4Call c{};
  c.x = x;
  c.q = q;
  c.scale = scale;
  c.zero = zero;
  c.out = out;
  c.M = M;
  c.N = N;
  c.K = K;
  c.group = (int)group;
  c.gated = gated;
  c.act = act;
  c.stream = static_cast<hipStream_t>(stream);
  c.dev = s.dev;
  return launch(c);
}

}  // namespace

extern "C" {

pgemm_status pgemm_fused_workspace(pgemm_fused_op op, int64_t M, int64_t N, int64_t K, int64_t *bytes) {
  if (!bytes) return PGEMM_ERR_NULL;
  const bool block = op == PGEMM_FUSED_GATED || op == PGEMM_FUSED_GATED_SAVE || op == PGEMM_FUSED_GATED_BWD;
  if (!block && op != PGEMM_FUSED_XENT && op != PGEMM_FUSED_XENT_BWD) return PGEMM_ERR_SHAPE;
  pgemm_status st = block ? check_gated(M, N, K, PGEMM_ACT_SILU) : check_xent(M, N, K);
  if (st != PGEMM_OK) return st;
  *bytes = block ? plan_gated(M, N, K, op == PGEMM_FUSED_GATED_BWD, op == PGEMM_FUSED_GATED_SAVE).bytes
                 : plan_xent(M, N, K, op == PGEMM_FUSED_XENT_BWD).bytes;
  return PGEMM_OK;
}

#define PGEMM_FUSED_ENTRIES(TYPE)                                                                                      \
  pgemm_status pgemm_##TYPE##_gated(const uint16_t *x, const uint16_t *w, uint16_t *h, float *saved, int64_t M,        \
                                    int64_t F, int64_t D, int act, void *stream) {                                     \
    return gated(gated_##TYPE, x, w, h, saved, M, F, D, act, stream);                                                  \
  }                                                                                                                    \
  pgemm_status pgemm_##TYPE##_gated_bwd(const uint16_t *dh, const uint16_t *x, const uint16_t *w, const float *saved,  \
                                        uint16_t *dx, uint16_t *dw, int64_t M, int64_t F, int64_t D, int act,          \
                                        void *stream) {                                                                \
    return gated_bwd(gated_bwd_##TYPE, dh, x, w, saved, dx, dw, M, F, D, act, stream);                                 \
  }                                                                                                                    \
  pgemm_status pgemm_##TYPE##_xent(const uint16_t *x, const uint16_t *w, const int64_t *target, float *loss,           \
                                   float *lse, int64_t M, int64_t V, int64_t D, int64_t ignore_index, void *stream) {  \
    return xent(xent_##TYPE, x, w, target, loss, lse, M, V, D, ignore_index, stream);                                  \
  }                                                                                                                    \
  pgemm_status pgemm_##TYPE##_xent_bwd(const float *dloss, int dloss_step, const uint16_t *x, const uint16_t *w,       \
                                       const int64_t *target, const float *lse, uint16_t *dx, uint16_t *dw, int64_t M, \
                                       int64_t V, int64_t D, int64_t ignore_index, void *stream) {                     \
    return xent_bwd(xent_bwd_##TYPE, dloss, dloss_step, x, w, target, lse, dx, dw, M, V, D, ignore_index, stream);     \
  }                                                                                                                    \
  pgemm_status pgemm_##TYPE##_q4(const uint16_t *x, const uint8_t *q, const uint16_t *scale, const uint8_t *zero,      \
                                 uint16_t *out, int64_t M, int64_t N, int64_t K, int64_t group, void *stream) {        \
    return q4(q4_##TYPE, x, q, scale, zero, out, M, N, K, group, false, PGEMM_ACT_SILU, stream);                       \
  }                                                                                                                    \
  pgemm_status pgemm_##TYPE##_q4_gated(const uint16_t *x, const uint8_t *q, const uint16_t *scale,                     \
                                       const uint8_t *zero, uint16_t *out, int64_t M, int64_t F, int64_t K,            \
                                       int64_t group, int act, void *stream) {                                         \
    return q4(q4_##TYPE, x, q, scale, zero, out, M, F, K, group, true, act, stream);                                   \
  }

PGEMM_FUSED_ENTRIES(f16)
PGEMM_FUSED_ENTRIES(bf16)

}  // extern "C"
