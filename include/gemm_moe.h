/*
 * gemm_moe.h -- C ABI of the mixture-of-experts layer of the gemm_f32 library
 * (MI355X, gfx950): the router, the chosen experts' products and their
 * weighted sum for a few tokens, as thin products over the weights of the
 * experts that were chosen.
 *
 * For each of T tokens (rows x of X):
 *   z[e]    = sum_h x[h] R[e][h]                      e < E, summed in 64 bits
 *   chosen  = the `top` experts of largest z, in falling order; of equal z the
 *             lower index first; a NaN counts as the lowest z here
 *   gate[s] = exp(z[chosen s]) / sum over all E of exp(z), or, with
 *             `renormalize`, over the chosen ones alone
 *   y       = sum_s gate[s] W2[e_s] u,   u[i] = silu(W1[e_s][i] . x) *
 *             (W1[e_s][I + i] . x),      silu(v) = v / (1 + exp(-v))
 *
 * Sums and u are held in fp32, and u's bits down to 2^-133 enter the second
 * product; y is rounded once to its format.  Results do not depend on timing.
 * A token whose row holds an infinity or a NaN may give NaN in its own row of Y
 * and gates, and no other's.  A NaN in a row of R does in the rows of the tokens
 * whose sum of exp(z) has it (with `renormalize`, those that choose its expert);
 * an infinity among W2's 16-bit weights may give NaN where it enters.
 *
 * Memory, streams and errors are as for gemm_f32 (gemm_f32.h): device
 * pointers owned by the caller, nothing allocated, asynchronous on `stream`,
 * argument errors returned before anything is enqueued, status codes
 * GEMM_F32_*.  Outputs and the workspace must not overlap inputs or one
 * another; calls that may overlap in time need workspaces of their own.
 */
#ifndef GEMM_MOE_H
#define GEMM_MOE_H

#ifdef __cplusplus
extern "C" {
#endif

/* What the experts' weights are: 16-bit codes of the tokens' format, row
 * pitches in elements; or MX matrices (gemm_mx.h), row pitches in bytes. */
#define GEMM_MOE_W16 0
#define GEMM_MOE_MX 1

#define GEMM_MOE_MAX_TOKENS 256
#define GEMM_MOE_MAX_EXPERTS 512
#define GEMM_MOE_MAX_TOP 16
#define GEMM_MOE_MAX_WIDTH (1 << 24)

/*
 * gemm_moe_workspace_bytes -- bytes of workspace a call needs, or -1 for sizes
 * that gemm_moe refuses.
 */
long long gemm_moe_workspace_bytes(int T, int E, int top, int H, int I);

/*
 * gemm_moe
 *   T         tokens, 0 .. GEMM_MOE_MAX_TOKENS (0: no-op)
 *   E, top    1 <= top <= E, top <= GEMM_MOE_MAX_TOP, E <= GEMM_MOE_MAX_EXPERTS
 *   H, I      the tokens' width and the experts' inner width, 1 ..
 *             GEMM_MOE_MAX_WIDTH
 *   X, R      T x H and E x H in `format` (GEMM_MIXED_BF16 or GEMM_MIXED_F16),
 *             2-byte aligned, pitches in elements
 *   W1        E * 2I rows of H values: expert e's rows from 2I e on, first I
 *             for the gate and then I for the other factor
 *   W2        E * H rows of I values: expert e's rows from H e on
 *   weights   GEMM_MOE_W16: W1 and W2 in `format`, 2-byte aligned, S1 and S2
 *             not read; GEMM_MOE_MX: MX codes, scales in S1 and S2
 *   Y         T x H in y_format: `format` or GEMM_MX_F32; element-aligned
 *   ids       T x top int, gates T x top float, contiguous; either may be NULL
 *   workspace 16-byte aligned, at least gemm_moe_workspace_bytes (else
 *             GEMM_F32_BAD_WORKSPACE); its content is neither read before it
 *             is written nor of use afterwards
 * Sizes outside these bounds: GEMM_F32_INVALID_DIM for negative ones and H or
 * I of 0, else GEMM_F32_BAD_ARG.
 */
int gemm_moe(int T, int E, int top, int H, int I, const void *X, int ldx, const void *R, int ldr,
             int format, const void *W1, int ld1, const unsigned char *S1, int lds1,
             const void *W2, int ld2, const unsigned char *S2, int lds2, int weights,
             int renormalize, void *Y, int ldy, int y_format, int *ids, float *gates,
             void *workspace, long long workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_MOE_H */
