// C ABI of the serving operators: argument checks, workspaces, dispatch by type.
//
// Arguments are checked before any HIP call, and nothing is enqueued for a
// call that is refused.
#include "api_checks.hpp"
#include "serve.hpp"

namespace {

using namespace pgemm;
using namespace pgemm::api;

bool off4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

template <typename Launch>
pgemm_status quant(Launch launch, const uint16_t *x, int8_t *q, float *scale, int64_t M, int64_t K, void *stream) {
  if (!dim(M) || !pitch(K)) return PGEMM_ERR_SHAPE;
  if (missing(x, M * K) || missing(q, M * K) || missing(scale, M)) return PGEMM_ERR_NULL;
  if (off16(x) || off16(q) || off16(scale)) return PGEMM_ERR_ALIGN;
  if (M == 0) return PGEMM_OK;
  Site s;
  pgemm_status st = s.open(stream, 0);
  if (st != PGEMM_OK) return st;
  return launch(QuantCall{x, q, scale, M, K, static_cast<hipStream_t>(stream)});
}

pgemm_status check_i8(int64_t M, int64_t N, int64_t K, bool gated, int act) {
  if (!dim(M) || !dim(N) || !dim(gated ? 2 * N : N) || K < 0 || K > kI8MaxK || !act_ok(act)) return PGEMM_ERR_SHAPE;
  if (!grid_fits(M, N) || per(N, 16) * 512 >= kMaxWorkItems) return PGEMM_ERR_SHAPE;
  return PGEMM_OK;
}

template <typename Launch>
pgemm_status i8(Launch launch, const void *x, const float *xs, const int8_t *w, const float *ws, uint16_t *out, int64_t M,
                int64_t N, int64_t K, bool gated, int act, void *stream) {
  pgemm_status st = check_i8(M, N, K, gated, act);
  if (st != PGEMM_OK) return st;
  if (missing(x, M * K) || missing(w, N * K) || missing(ws, N) || missing(out, M * N)) return PGEMM_ERR_NULL;
  if (off16(x) || off16(xs) || off16(w) || off16(ws) || off16(out)) return PGEMM_ERR_ALIGN;
  if (M == 0 || N == 0) return PGEMM_OK;
  Site s;
  st = s.open(stream, plan_i8(M, N, K, gated, xs != nullptr).bytes);
  if (st != PGEMM_OK) return st;
  I8Call c{};
  if (xs)
    c.q = static_cast<const int8_t *>(x);
  else
    c.x = static_cast<const uint16_t *>(x);
  c.xs = xs;
  c.w = w;
  c.ws = ws;
  c.out = out;
  c.M = M;
  c.N = N;
  c.K = K;
  c.gated = gated;
  c.act = act;
  c.workspace = s.ws;
  c.stream = static_cast<hipStream_t>(stream);
  c.dev = s.dev;
  return launch(c);
}

pgemm_status check_moe(int64_t M, int64_t E, int64_t D, int64_t F, int64_t top_k) {
  if (M < 0 || M >= kMoeMaxTokens || E < 1 || E > kMoeMaxExperts || !pitch(D) || F < 0 || F > kMoeMaxHidden || top_k < 1 ||
      top_k > kMoeMaxTop || top_k > E)
    return PGEMM_ERR_SHAPE;
  return PGEMM_OK;
}

template <typename Launch>
pgemm_status moe(Launch launch, const uint16_t *x, const uint16_t *router, const uint16_t *w, const uint16_t *down,
                 uint16_t *y, int32_t *experts, float *weights, int64_t M, int64_t E, int64_t D, int64_t F, int64_t top_k,
                 int normalize, int act, void *stream) {
  pgemm_status st = check_moe(M, E, D, F, top_k);
  if (st != PGEMM_OK) return st;
  if (!act_ok(act) || (normalize != 0 && normalize != 1)) return PGEMM_ERR_SHAPE;
  if (missing(x, M * D) || missing(router, D) || missing(w, F * D) || missing(down, F * D) || missing(y, M * D))
    return PGEMM_ERR_NULL;
  if (off16(x) || off16(router) || off16(w) || off16(down) || off16(y) || off16(experts) || off16(weights))
    return PGEMM_ERR_ALIGN;
  if (M == 0) return PGEMM_OK;
  Site s;
  st = s.open(stream, plan_moe(M, E, D, F, top_k).bytes);
  if (st != PGEMM_OK) return st;
  MoeCall c{};
  c.x = x;
  c.router = router;
  c.w = w;
  c.down = down;
  c.y = y;
  c.experts = experts;
  c.weights = weights;
  c.M = M;
  c.E = E;
  c.D = D;
  c.F = F;
  c.top_k = top_k;
  c.normalize = normalize != 0;
  c.act = act;
  c.workspace = s.ws;
  c.stream = static_cast<hipStream_t>(stream);
  c.dev = s.dev;
  return launch(c);
}

template <typename Launch>
pgemm_status sample(Launch launch, const uint16_t *logits, const float *u, const float *temperature, const int32_t *top_k,
                    const float *top_p, const float *min_p, int shared, int64_t *token, int64_t M, int64_t V, void *stream) {
  if (!dim(M) || V < 0 || V > (int64_t)1 << 30 || shared < 0 || shared > 15) return PGEMM_ERR_SHAPE;
  if (missing(logits, M * V) || missing(u, M) || missing(token, M)) return PGEMM_ERR_NULL;
  if (off16(logits) || off16(token) || off4(u) || off4(temperature) || off4(top_k) || off4(top_p) || off4(min_p))
    return PGEMM_ERR_ALIGN;
  if (M == 0) return PGEMM_OK;
  Site s;
  pgemm_status st = s.open(stream, 0);
  if (st != PGEMM_OK) return st;
  return launch(SampleCall{logits, u, temperature, top_k, top_p, min_p, shared, token, M, V,
                           static_cast<hipStream_t>(stream), s.dev});
}

}  // namespace

extern "C" {

pgemm_status pgemm_i8_workspace(int64_t M, int64_t N, int64_t K, int gated, int quantized, int64_t *bytes) {
  if (!bytes) return PGEMM_ERR_NULL;
  pgemm_status st = check_i8(M, N, K, gated != 0, PGEMM_ACT_SILU);
  if (st != PGEMM_OK) return st;
  *bytes = M == 0 || N == 0 ? 0 : plan_i8(M, N, K, gated != 0, quantized != 0).bytes;
  return PGEMM_OK;
}

pgemm_status pgemm_moe_workspace(int64_t M, int64_t E, int64_t D, int64_t F, int64_t top_k, int64_t *bytes) {
  if (!bytes) return PGEMM_ERR_NULL;
  pgemm_status st = check_moe(M, E, D, F, top_k);
  if (st != PGEMM_OK) return st;
  *bytes = M == 0 ? 0 : plan_moe(M, E, D, F, top_k).bytes;
  return PGEMM_OK;
}

#define PGEMM_SERVE_ENTRIES(TYPE)                                                                                         \
  pgemm_status pgemm_##TYPE##_quant_i8(const uint16_t *x, int8_t *q, float *scale, int64_t M, int64_t K, void *stream) {  \
    return quant(quant_i8_##TYPE, x, q, scale, M, K, stream);                                                             \
  }                                                                                                                       \
  pgemm_status pgemm_##TYPE##_i8(const void *x, const float *xs, const int8_t *w, const float *ws, uint16_t *out,         \
                                 int64_t M, int64_t N, int64_t K, void *stream) {                                         \
    return i8(i8_##TYPE, x, xs, w, ws, out, M, N, K, false, PGEMM_ACT_SILU, stream);                                      \
  }                                                                                                                       \
  pgemm_status pgemm_##TYPE##_i8_gated(const void *x, const float *xs, const int8_t *w, const float *ws, uint16_t *out,   \
                                       int64_t M, int64_t F, int64_t K, int act, void *stream) {                          \
    return i8(i8_##TYPE, x, xs, w, ws, out, M, F, K, true, act, stream);                                                  \
  }                                                                                                                       \
  pgemm_status pgemm_##TYPE##_moe(const uint16_t *x, const uint16_t *router, const uint16_t *w, const uint16_t *down,     \
                                  uint16_t *y, int32_t *experts, float *weights, int64_t M, int64_t E, int64_t D,         \
                                  int64_t F, int64_t top_k, int normalize, int act, void *stream) {                       \
    return moe(moe_##TYPE, x, router, w, down, y, experts, weights, M, E, D, F, top_k, normalize, act, stream);           \
  }                                                                                                                       \
  pgemm_status pgemm_##TYPE##_sample(const uint16_t *logits, const float *u, const float *temperature,                    \
                                     const int32_t *top_k, const float *top_p, const float *min_p, int shared,            \
                                     int64_t *token, int64_t M, int64_t V, void *stream) {                                \
    return sample(sample_##TYPE, logits, u, temperature, top_k, top_p, min_p, shared, token, M, V, stream);               \
  }

PGEMM_SERVE_ENTRIES(f16)
PGEMM_SERVE_ENTRIES(bf16)

}  // extern "C"
