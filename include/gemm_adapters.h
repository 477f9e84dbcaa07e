/*
 * gemm_adapters.h -- C ABI of a shared projection with low-rank adapters of many
 * requests of the gemm_f32 library (MI355X, gfx950).
 *
 * For each of T rows x of X, r = ids[t]:
 *   y = W x + scales[r] B[r] (A[r] x)      r in 0 .. count - 1
 *   y = W x                                any other r: a row without an adapter
 * Sums are held in fp32, and y is rounded once.  scales[r] A[r] x is rounded to the
 * precision of `format` on its way into the second product (an error of the size of
 * the result's own), not to its range: in fp16 each row's values, in groups of up to
 * 64 ranks, have an exponent of their own (one below 2^-28 of its group's largest may
 * be lost).  Results do not depend on timing.  An infinity or a NaN reaches the rows
 * that it enters alone: a row's own values, W's, and its own adapter's.
 *
 * Memory, streams and errors are as for gemm_f32 (gemm_f32.h): device
 * pointers owned by the caller, nothing allocated, asynchronous on `stream`,
 * argument errors returned before anything is enqueued, status codes
 * GEMM_F32_*.  Outputs and the workspace must not overlap inputs or one
 * another; calls that may overlap in time need workspaces of their own.
 */
#ifndef GEMM_ADAPTERS_H
#define GEMM_ADAPTERS_H

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_ADAPTERS_MAX_ROWS (1 << 22)
#define GEMM_ADAPTERS_MAX_WIDTH (1 << 17)
#define GEMM_ADAPTERS_MAX_RANK 512
#define GEMM_ADAPTERS_MAX_COUNT 511

/* Bytes of workspace that a call needs, or -1 for sizes that it refuses. */
long long gemm_adapters_workspace_bytes(int T, int N, int K, int R, int count);

/*
 * gemm_adapters
 *   T         rows, 0 .. GEMM_ADAPTERS_MAX_ROWS (0: no-op)
 *   N, K      1 .. GEMM_ADAPTERS_MAX_WIDTH
 *   R         the adapters' rank, 1 .. GEMM_ADAPTERS_MAX_RANK
 *   count     adapters, 0 .. GEMM_ADAPTERS_MAX_COUNT (0: A and B are not read)
 *   X, W, Y   T x K, N x K and T x N in `format` (GEMM_MIXED_BF16 or
 *             GEMM_MIXED_F16), 2-byte aligned, pitches in elements.  (Of more than
 *             2^31 bytes, X or W, many rows take nearly twice as long.)
 *   A         count * R rows of K values: adapter r's rows from R r on
 *   B         count * N rows of R values: adapter r's rows from N r on
 *   ids       T int
 *   scales    count float, or NULL: 1 each
 *   workspace 16-byte aligned, at least gemm_adapters_workspace_bytes (else
 *             GEMM_F32_BAD_WORKSPACE); its content is neither read before it
 *             is written nor of use afterwards
 * Sizes outside these bounds: GEMM_F32_INVALID_DIM for negative ones and N, K or
 * R of 0, else GEMM_F32_BAD_ARG.
 */
int gemm_adapters(int T, int N, int K, int R, int count, const void *X, int ldx, const void *W,
                  int ldw, const void *A, int lda, const void *B, int ldb, const int *ids,
                  const float *scales, int format, void *Y, int ldy, void *workspace,
                  long long workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_ADAPTERS_H */
