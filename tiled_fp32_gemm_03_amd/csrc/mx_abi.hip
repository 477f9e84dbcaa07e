// C-ABI front end of the MX operators (gemm_mx.h): argument checks, in the
// order sizes, row pitches, formats, pointers, then one launch.  Every error
// is returned before anything is enqueued.
#include "gemm_f32.h"
#include "gemm_internal.hpp"
#include "gemm_mixed.h"
#include "gemm_moe.h"
#include "gemm_mx.h"
#include "mx_internal.hpp"

using namespace gemm_f32_impl;

static_assert(kBf16 == GEMM_MIXED_BF16 && kF16 == GEMM_MIXED_F16 && kF32 == GEMM_MX_F32 &&
                  kAlongRows == GEMM_MX_ROWS && kAlongColumns == GEMM_MX_COLUMNS,
              "constants of mx_plan.hpp and the headers differ");
static_assert(kMoeMaxTokens == GEMM_MOE_MAX_TOKENS && kMoeMaxExperts == GEMM_MOE_MAX_EXPERTS &&
                  kMoeMaxTop == GEMM_MOE_MAX_TOP && kMoeMaxWidth == GEMM_MOE_MAX_WIDTH,
              "bounds of mx_plan.hpp and gemm_moe.h differ");

extern "C" long long gemm_mx_code_bytes(int K) { return K < 0 ? 0 : mx_code_bytes(K); }
extern "C" long long gemm_mx_scale_bytes(int K) { return K < 0 ? 0 : mx_scale_bytes(K); }

namespace {

// The checks of both conversions.  `plain` is X or Y.
int convert_check(int rows, int K, const void *plain, int ldx, int format, int along,
                  const void *codes, int ld, const void *scales, int lds) {
  int rc = check_shape(rows, rows, K);
  if (rc != GEMM_F32_OK) return rc;
  if (!is_format(format) || (along != kAlongRows && along != kAlongColumns))
    return GEMM_F32_BAD_ARG;
  const int len = along == kAlongRows ? K : rows;
  if (ldx < (len > 1 ? len : 1)) return GEMM_F32_INVALID_LD;
  rc = check_mx_ld(K, ld, lds);
  if (rc != GEMM_F32_OK) return rc;
  if (rows == 0 || K == 0) return GEMM_F32_OK;
  rc = check_plain_pointer(plain, format);
  return rc != GEMM_F32_OK ? rc : check_mx_pointers(codes, scales);
}

}  // namespace

extern "C" int gemm_mx_quantize(int rows, int K, const void *X, int ldx, int format, int along,
                                unsigned char *codes, int ld, unsigned char *scales, int lds,
                                void *stream) {
  const int rc = convert_check(rows, K, X, ldx, format, along, codes, ld, scales, lds);
  if (rc != GEMM_F32_OK || rows == 0 || K == 0) return rc;
  const MxConvert c{rows, K, X, nullptr, ldx, codes, ld, scales, lds};
  return launch_status(launch_mx_quantize(format, along, c, static_cast<hipStream_t>(stream)),
                       "mx quantize");
}

extern "C" int gemm_mx_dequantize(int rows, int K, const unsigned char *codes, int ld,
                                  const unsigned char *scales, int lds, void *Y, int ldy,
                                  int format, int along, void *stream) {
  const int rc = convert_check(rows, K, Y, ldy, format, along, codes, ld, scales, lds);
  if (rc != GEMM_F32_OK || rows == 0 || K == 0) return rc;
  const MxConvert c{rows, K, nullptr, Y, ldy, const_cast<unsigned char *>(codes), ld,
                    const_cast<unsigned char *>(scales), lds};
  return launch_status(launch_mx_dequantize(format, along, c, static_cast<hipStream_t>(stream)),
                       "mx dequantize");
}

// ---- products ----------------------------------------------------------------

namespace {

int mx_resolve(int config, int M, int N, int K, int *out) {
  if (config < -1 || config >= mx_num_entries()) return GEMM_F32_BAD_CONFIG;
  *out = config == -1 ? mx_choose(M, N, K) : config;
  return GEMM_F32_OK;
}

int check_ldc(int N, int ldc) { return ldc < (N > 1 ? N : 1) ? kInvalidLd : kOk; }

}  // namespace

extern "C" int gemm_mx(int M, int N, int K, const unsigned char *A, int lda,
                       const unsigned char *SA, int ldsa, const unsigned char *B, int ldb,
                       const unsigned char *SB, int ldsb, void *C, int ldc, int c_format,
                       int config, void *stream) {
  int rc = check_shape(M, N, K);
  if (rc == kOk) rc = check_mx_ld(K, lda, ldsa);
  if (rc == kOk) rc = check_mx_ld(K, ldb, ldsb);
  if (rc == kOk) rc = check_ldc(N, ldc);
  if (rc == kOk && !is_format(c_format)) rc = kBadArg;
  int entry = 0;
  if (rc == kOk) rc = mx_resolve(config, M, N, K, &entry);
  if (rc != kOk || M == 0 || N == 0) return rc;
  rc = check_plain_pointer(C, c_format);
  if (rc == kOk && K > 0) rc = check_mx_pointers(A, SA);
  if (rc == kOk && K > 0) rc = check_mx_pointers(B, SB);
  if (rc != kOk) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (K == 0) return launch_status(launch_mx_zero(C, M, N, ldc, c_format, s), "zero fill");
  const MxProblem p{M, N, K, {A, lda, SA, ldsa}, {B, ldb, SB, ldsb}, C, ldc, c_format};
  return launch_status(launch_mx_gemm(entry, p, s), "mx product");
}

extern "C" int gemm_mx_num_configs(void) { return mx_num_entries(); }

extern "C" int gemm_mx_tile(int config, int M, int N, int K, int *BM, int *BN, int *BK,
                            int *threads, int *chosen_config) {
  int rc = check_shape(M, N, K);
  int entry = 0;
  if (rc == kOk) rc = mx_resolve(config, M, N, K, &entry);
  if (rc != kOk) return rc;
  const MxEntry &e = mx_entry(entry);
  if (BM) *BM = e.BM;
  if (BN) *BN = e.BN;
  if (BK) *BK = e.BK;
  if (threads) *threads = e.threads;
  if (chosen_config) *chosen_config = entry;
  return GEMM_F32_OK;
}

extern "C" int gemm_mx_a16(int M, int N, int K, const void *A, int lda, int a_format,
                           const unsigned char *B, int ldb, const unsigned char *SB, int ldsb,
                           void *C, int ldc, int c_format, void *stream) {
  int rc = check_shape(M, N, K);
  if (rc == kOk && lda < (K > 1 ? K : 1)) rc = kInvalidLd;
  if (rc == kOk) rc = check_mx_ld(K, ldb, ldsb);
  if (rc == kOk) rc = check_ldc(N, ldc);
  if (rc == kOk && (!is_format(c_format) || (a_format != kBf16 && a_format != kF16))) rc = kBadArg;
  if (rc != kOk || M == 0 || N == 0) return rc;
  rc = check_plain_pointer(C, c_format);
  if (rc == kOk && K > 0) rc = check_plain_pointer(A, a_format);
  if (rc == kOk && K > 0) rc = check_mx_pointers(B, SB);
  if (rc != kOk) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (K == 0) return launch_status(launch_mx_zero(C, M, N, ldc, c_format, s), "zero fill");
  const MxA16Problem p{M, N, K, static_cast<const uint16_t *>(A), lda, a_format,
                       {B, ldb, SB, ldsb}, C, ldc, c_format};
  return launch_status(launch_mx_a16(p, s), "mx 16-bit product");
}

// ---- the mixture-of-experts layer ----------------------------------------------

extern "C" long long gemm_moe_workspace_bytes(int T, int E, int top, int H, int I) {
  return moe_check_sizes(T, E, top, H, I) == kOk ? moe_space(T, E, top, H, I).bytes : -1;
}

extern "C" int gemm_moe(int T, int E, int top, int H, int I, const void *X, int ldx,
                        const void *R, int ldr, int format, const void *W1, int ld1,
                        const unsigned char *S1, int lds1, const void *W2, int ld2,
                        const unsigned char *S2, int lds2, int weights, int renormalize, void *Y,
                        int ldy, int y_format, int *ids, float *gates, void *workspace,
                        long long workspace_bytes, void *stream) {
  int rc = moe_check_sizes(T, E, top, H, I);
  if (rc != kOk) return rc;
  if ((format != kBf16 && format != kF16) || (y_format != format && y_format != kF32) ||
      (weights != GEMM_MOE_W16 && weights != GEMM_MOE_MX))
    return kBadArg;
  const bool mx = weights == GEMM_MOE_MX;
  if (ldx < H || ldr < H || ldy < H) return kInvalidLd;
  if (mx) {
    rc = check_mx_ld(H, ld1, lds1);
    if (rc == kOk) rc = check_mx_ld(I, ld2, lds2);
    if (rc != kOk) return rc;
  } else if (ld1 < H || ld2 < I) {
    return kInvalidLd;
  }
  if (T == 0) return kOk;
  rc = check_plain_pointer(X, format);
  if (rc == kOk) rc = check_plain_pointer(R, format);
  if (rc == kOk) rc = check_plain_pointer(Y, y_format);
  if (rc == kOk) rc = mx ? check_mx_pointers(W1, S1) : check_plain_pointer(W1, format);
  if (rc == kOk) rc = mx ? check_mx_pointers(W2, S2) : check_plain_pointer(W2, format);
  if (rc == kOk && ids != nullptr) rc = check_plain_pointer(ids, kF32);
  if (rc == kOk && gates != nullptr) rc = check_plain_pointer(gates, kF32);
  if (rc != kOk) return rc;
  const MoeSpace at = moe_space(T, E, top, H, I);
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15) != 0 ||
      workspace_bytes < at.bytes)
    return GEMM_F32_BAD_WORKSPACE;
  const MoeProblem p{T, E, top, H, I, static_cast<const uint16_t *>(X), ldx,
                     static_cast<const uint16_t *>(R), ldr, format,
                     static_cast<const unsigned char *>(W1), mx ? ld1 : 2LL * ld1, S1, lds1,
                     static_cast<const unsigned char *>(W2), mx ? ld2 : 2LL * ld2, S2, lds2,
                     mx, renormalize != 0, Y, ldy, y_format, ids, gates,
                     static_cast<unsigned char *>(workspace), at, nullptr, nullptr};
  return launch_status(launch_moe(p, static_cast<hipStream_t>(stream)), "moe");
}
