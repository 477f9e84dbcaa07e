// C-ABI front end of routing (gemm_route.h), the experts' products
// (gemm_experts.h) and adapters (gemm_adapters.h): argument checks, in the order sizes, row pitches, formats,
// pointers, workspace, then the launches.  Every error is returned before
// anything is enqueued.
#include "experts_internal.hpp"
#include "gemm_adapters.h"
#include "gemm_experts.h"
#include "gemm_f32.h"
#include "gemm_internal.hpp"
#include "gemm_mixed.h"
#include "gemm_moe.h"
#include "gemm_mx.h"
#include "gemm_route.h"
#include "mx_internal.hpp"
#include "route_internal.hpp"

using namespace gemm_f32_impl;

static_assert(kRouteMaxTokens == GEMM_ROUTE_MAX_TOKENS && kRouteMaxExperts == GEMM_ROUTE_MAX_EXPERTS &&
                  kRouteMaxTop == GEMM_ROUTE_MAX_TOP && kRouteMaxGroups == GEMM_ROUTE_MAX_GROUPS &&
                  kSoftmax == GEMM_ROUTE_SOFTMAX && kSigmoid == GEMM_ROUTE_SIGMOID &&
                  kGroupMax == GEMM_ROUTE_MAX && kGroupTop2 == GEMM_ROUTE_TOP2,
              "constants of experts_plan.hpp and gemm_route.h differ");
static_assert(kExpertsMaxTokens == GEMM_EXPERTS_MAX_TOKENS &&
                  kExpertsMaxWidth == GEMM_EXPERTS_MAX_WIDTH,
              "bounds of experts_plan.hpp and gemm_experts.h differ");
static_assert(kAdaptersMaxRows == GEMM_ADAPTERS_MAX_ROWS &&
                  kAdaptersMaxWidth == GEMM_ADAPTERS_MAX_WIDTH &&
                  kAdaptersMaxRank == GEMM_ADAPTERS_MAX_RANK &&
                  kAdaptersMaxCount == GEMM_ADAPTERS_MAX_COUNT,
              "bounds of experts_plan.hpp and gemm_adapters.h differ");

namespace {

bool is_16(int format) { return format == kBf16 || format == kF16; }
// A pointer to 4-byte values.
int check_words(const void *p) { return check_plain_pointer(p, kF32); }

}  // namespace

extern "C" int gemm_moe_route(int T, int E, int top, const void *Z, int ldz, int format, int score,
                              const float *bias, int groups, int top_groups, int group_score,
                              int renormalize, float scale, int *ids, float *gates, void *stream) {
  int rc = route_check_sizes(T, E, top);
  if (rc != kOk) return rc;
  if (groups < 1 || groups > kRouteMaxGroups || E % groups != 0 || top_groups < 1 ||
      top_groups > groups || top > top_groups * (E / groups))
    return kBadArg;
  if (ldz < E) return kInvalidLd;
  if (!is_format(format) || (score != kSoftmax && score != kSigmoid) ||
      (group_score != kGroupMax && group_score != kGroupTop2) || !(scale - scale == 0.f))
    return kBadArg;
  if (T == 0) return kOk;
  rc = check_plain_pointer(Z, format);
  if (rc == kOk && bias) rc = check_words(bias);
  if (rc == kOk) rc = check_words(ids);
  if (rc == kOk) rc = check_words(gates);
  if (rc != kOk) return rc;
  RouteProblem p{};
  p.T = T, p.E = E, p.top = top, p.Z = Z, p.ldz = ldz, p.format = format, p.score = score;
  p.bias = bias, p.groups = groups, p.top_groups = top_groups, p.group_score = group_score;
  p.renormalize = renormalize != 0, p.scale = scale, p.ids = ids, p.gates = gates;
  return launch_status(launch_route(p, static_cast<hipStream_t>(stream)), "route");
}

extern "C" int gemm_moe_route_backward(int T, int E, int top, const float *dgates, const void *Z,
                                       int ldz, int format, int score, int renormalize, float scale,
                                       const int *ids, void *dZ, int lddz, void *stream) {
  int rc = route_check_sizes(T, E, top);
  if (rc != kOk) return rc;
  if (ldz < E || lddz < E) return kInvalidLd;
  if (!is_format(format) || (score != kSoftmax && score != kSigmoid) || !(scale - scale == 0.f))
    return kBadArg;
  if (T == 0) return kOk;
  rc = check_words(dgates);
  if (rc == kOk) rc = check_plain_pointer(Z, format);
  if (rc == kOk) rc = check_words(ids);
  if (rc == kOk) rc = check_plain_pointer(dZ, format);
  if (rc != kOk) return rc;
  RouteProblem p{};
  p.T = T, p.E = E, p.top = top, p.Z = Z, p.ldz = ldz, p.format = format, p.score = score;
  p.renormalize = renormalize != 0, p.scale = scale, p.given = ids, p.dgates = dgates;
  p.dZ = dZ, p.lddz = lddz;
  return launch_status(launch_route_backward(p, static_cast<hipStream_t>(stream)),
                       "route backward");
}

// ---- the experts' products -------------------------------------------------------

namespace {

long long experts_bytes(int T, int E, int top, int H, int I, bool backward) {
  // (of smaller tiles: they need the most)
  const long long tiles = experts_space(T, E, top, H, I, 128, backward).bytes;
  if (backward) return tiles;
  long long most = tiles;
  if (T <= kMoeMaxTokens && moe_space(T, E, top, H, I).bytes > most)
    most = moe_space(T, E, top, H, I).bytes;
  return most;
}

bool bad_workspace(const void *ws, long long bytes, long long need) {
  return ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 15) != 0 || bytes < need;
}

}  // namespace

extern "C" long long gemm_experts_workspace_bytes(int T, int E, int top, int H, int I,
                                                  int backward) {
  if (experts_check_sizes(T, E, top, H, I) != kOk) return -1;
  return experts_bytes(T, E, top, H, I, backward != 0);
}

extern "C" int gemm_experts(int T, int E, int top, int H, int I, const void *X, int ldx,
                            const int *ids, const float *gates, int format, const void *W1, int ld1,
                            const unsigned char *S1, int lds1, const void *W2, int ld2,
                            const unsigned char *S2, int lds2, int weights, void *Y, int ldy,
                            float *saved, void *workspace, long long workspace_bytes,
                            void *stream) {
  int rc = experts_check_sizes(T, E, top, H, I);
  if (rc != kOk) return rc;
  if (!is_16(format) || (weights != GEMM_MOE_W16 && weights != GEMM_MOE_MX)) return kBadArg;
  const bool mx = weights == GEMM_MOE_MX;
  if (mx && (T > kMoeMaxTokens || saved != nullptr)) return kBadArg;
  if (ldx < H || ldy < H) return kInvalidLd;
  if (mx) {
    rc = check_mx_ld(H, ld1, lds1);
    if (rc == kOk) rc = check_mx_ld(I, ld2, lds2);
    if (rc != kOk) return rc;
  } else if (ld1 < H || ld2 < I) {
    return kInvalidLd;
  }
  if (T == 0) return kOk;
  rc = check_plain_pointer(X, format);
  if (rc == kOk) rc = check_words(ids);
  if (rc == kOk) rc = check_words(gates);
  if (rc == kOk) rc = mx ? check_mx_pointers(W1, S1) : check_plain_pointer(W1, format);
  if (rc == kOk) rc = mx ? check_mx_pointers(W2, S2) : check_plain_pointer(W2, format);
  if (rc == kOk) rc = check_plain_pointer(Y, format);
  if (rc == kOk && saved) rc = check_words(saved);
  if (rc != kOk) return rc;
  if (bad_workspace(workspace, workspace_bytes, experts_bytes(T, E, top, H, I, false)))
    return GEMM_F32_BAD_WORKSPACE;
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (mx || (saved == nullptr && experts_thin(T, E, top))) {
    const MoeProblem p{T, E, top, H, I, static_cast<const uint16_t *>(X), ldx, nullptr, 0, format,
                       static_cast<const unsigned char *>(W1), mx ? ld1 : 2LL * ld1, S1, lds1,
                       static_cast<const unsigned char *>(W2), mx ? ld2 : 2LL * ld2, S2, lds2, mx,
                       0, Y, ldy, format, nullptr, nullptr, ws, moe_space(T, E, top, H, I), ids,
                       gates};
    return launch_status(launch_moe(p, s), "experts");
  }
  ExpertsProblem p{};
  p.T = T, p.E = E, p.top = top, p.H = H, p.I = I, p.format = format;
  p.X = static_cast<const uint16_t *>(X), p.ldx = ldx, p.ids = ids, p.gates = gates;
  p.W1 = static_cast<const uint16_t *>(W1), p.ld1 = ld1;
  p.W2 = static_cast<const uint16_t *>(W2), p.ld2 = ld2;
  p.Y = static_cast<uint16_t *>(Y), p.ldy = ldy, p.saved = saved, p.ws = ws;
  return launch_status(launch_experts_forward(p, s), "experts");
}

extern "C" int gemm_experts_backward(int T, int E, int top, int H, int I, const void *dY, int lddy,
                                     const void *X, int ldx, const int *ids, const float *gates,
                                     int format, const void *W1, int ld1, const void *W2, int ld2,
                                     const float *saved, void *dX, int lddx, float *dgates,
                                     void *dW1, int lddw1, void *dW2, int lddw2, void *workspace,
                                     long long workspace_bytes, void *stream) {
  int rc = experts_check_sizes(T, E, top, H, I);
  if (rc != kOk) return rc;
  if (!is_16(format)) return kBadArg;
  if (lddy < H || ldx < H || ld1 < H || ld2 < I || (dX && lddx < H) || (dW1 && lddw1 < H) ||
      (dW2 && lddw2 < I))
    return kInvalidLd;
  if (T > 0) {
    rc = check_plain_pointer(dY, format);
    if (rc == kOk) rc = check_plain_pointer(X, format);
    if (rc == kOk) rc = check_words(ids);
    if (rc == kOk) rc = check_words(gates);
    if (rc == kOk) rc = check_plain_pointer(W1, format);
    if (rc == kOk) rc = check_plain_pointer(W2, format);
    if (rc == kOk) rc = check_words(saved);
    if (rc == kOk && dX) rc = check_plain_pointer(dX, format);
    if (rc == kOk && dgates) rc = check_words(dgates);
    if (rc != kOk) return rc;
  }
  if (dW1) rc = check_plain_pointer(dW1, format);
  if (rc == kOk && dW2) rc = check_plain_pointer(dW2, format);
  if (rc != kOk) return rc;
  if (bad_workspace(workspace, workspace_bytes, experts_bytes(T, E, top, H, I, true)))
    return GEMM_F32_BAD_WORKSPACE;
  ExpertsProblem p{};
  p.T = T, p.E = E, p.top = top, p.H = H, p.I = I, p.format = format;
  p.X = static_cast<const uint16_t *>(X), p.ldx = ldx, p.ids = ids, p.gates = gates;
  p.W1 = static_cast<const uint16_t *>(W1), p.ld1 = ld1;
  p.W2 = static_cast<const uint16_t *>(W2), p.ld2 = ld2;
  p.saved = const_cast<float *>(saved), p.dY = static_cast<const uint16_t *>(dY), p.lddy = lddy;
  p.dX = static_cast<uint16_t *>(dX), p.lddx = lddx, p.dgates = dgates;
  p.dW1 = static_cast<uint16_t *>(dW1), p.lddw1 = lddw1;
  p.dW2 = static_cast<uint16_t *>(dW2), p.lddw2 = lddw2;
  p.ws = static_cast<unsigned char *>(workspace);
  return launch_status(launch_experts_backward(p, static_cast<hipStream_t>(stream)),
                       "experts backward");
}

// ---- adapters ----------------------------------------------------------------------

extern "C" long long gemm_adapters_workspace_bytes(int T, int N, int K, int R, int count) {
  return adapters_check_sizes(T, N, K, R, count) == kOk ? adapters_space(T, N, K, R, count).bytes
                                                        : -1;
}

extern "C" int gemm_adapters(int T, int N, int K, int R, int count, const void *X, int ldx,
                             const void *W, int ldw, const void *A, int lda, const void *B, int ldb,
                             const int *ids, const float *scales, int format, void *Y, int ldy,
                             void *workspace, long long workspace_bytes, void *stream) {
  int rc = adapters_check_sizes(T, N, K, R, count);
  if (rc != kOk) return rc;
  if (!is_16(format)) return kBadArg;
  if (ldx < K || ldw < K || ldy < N || (count > 0 && (lda < K || ldb < R))) return kInvalidLd;
  if (T == 0) return kOk;
  rc = check_plain_pointer(X, format);
  if (rc == kOk) rc = check_plain_pointer(W, format);
  if (rc == kOk && count > 0) rc = check_plain_pointer(A, format);
  if (rc == kOk && count > 0) rc = check_plain_pointer(B, format);
  if (rc == kOk) rc = check_words(ids);
  if (rc == kOk && scales) rc = check_words(scales);
  if (rc == kOk) rc = check_plain_pointer(Y, format);
  if (rc != kOk) return rc;
  const AdaptersSpace at = adapters_space(T, N, K, R, count);
  if (bad_workspace(workspace, workspace_bytes, at.bytes)) return GEMM_F32_BAD_WORKSPACE;
  const AdaptersProblem p{T, N, K, R, count, format, static_cast<const uint16_t *>(X), ldx,
                          static_cast<const uint16_t *>(W), ldw, static_cast<const uint16_t *>(A),
                          lda, static_cast<const uint16_t *>(B), ldb, ids, scales,
                          static_cast<uint16_t *>(Y), ldy, static_cast<unsigned char *>(workspace),
                          at};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return launch_status(adapters_thin(T, N, K) ? launch_adapters_thin(p, s) : launch_adapters_tiles(p, s),
                       "adapters");
}
