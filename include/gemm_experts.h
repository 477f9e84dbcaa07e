/*
 * gemm_experts.h -- C ABI of the experts' products of a mixture-of-experts layer
 * of the gemm_f32 library (MI355X, gfx950), for a choice of experts made before
 * (gemm_route.h) and any number of tokens, with their gradients.  (gemm_moe.h has
 * the layer with its own router for a few tokens.)
 *
 * For each of T tokens (rows x of X), e = ids[t][s]:
 *   h = W1[e] x,   u[i] = silu(h[i]) h[I + i],   silu(v) = v / (1 + exp(-v))
 *   y = sum_s gates[t][s] W2[e] u
 * An id outside 0 .. E - 1 is a choice that was dropped: it adds nothing, and its
 * gate's gradient is 0.  The same id twice in a row counts twice.
 *
 * Sums are held in fp32, and results do not depend on timing.  u and, in the
 * backward pass, gates[t][s] u and the gradient of h are kept in `format` between
 * the products: in fp16 values past 65,504 become infinite, and those below 2^-14 lose
 * bits.  Without `saved`, up to GEMM_MOE_MAX_TOKENS tokens and 6 choices to an expert
 * (T top <= 6 E, and always for MX weights), u is kept in fp32.  So with `saved`, or
 * among more tokens, a token's result may differ in its last bits, and in fp16 may be
 * infinite where it is not otherwise.
 * An infinity or a NaN reaches what is computed from it: a token's own rows, and
 * the weights' gradients of its experts.
 *
 * Memory, streams and errors are as for gemm_f32 (gemm_f32.h): device
 * pointers owned by the caller, nothing allocated, asynchronous on `stream`,
 * argument errors returned before anything is enqueued, status codes
 * GEMM_F32_*.  Outputs and the workspace must not overlap inputs or one
 * another; calls that may overlap in time need workspaces of their own.
 */
#ifndef GEMM_EXPERTS_H
#define GEMM_EXPERTS_H

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_EXPERTS_MAX_TOKENS (1 << 22)
#define GEMM_EXPERTS_MAX_WIDTH (1 << 17)

/*
 * Bytes of workspace that a call needs, or -1 for sizes that it refuses.
 * `backward`: 0 for gemm_experts, 1 for gemm_experts_backward.
 */
long long gemm_experts_workspace_bytes(int T, int E, int top, int H, int I, int backward);

/*
 * gemm_experts
 *   T         0 .. GEMM_EXPERTS_MAX_TOKENS (0: no-op)
 *   E, top    1 .. 512 (GEMM_MOE_MAX_EXPERTS) and 1 .. 16 (GEMM_MOE_MAX_TOP)
 *   H, I      1 .. GEMM_EXPERTS_MAX_WIDTH
 *   X         T x H in `format` (GEMM_MIXED_BF16 or GEMM_MIXED_F16), 2-byte
 *             aligned, pitches in elements.  (Of more than 2^31 bytes, 2 T ldx, a call
 *             takes half as long again, and so with dY; two calls do not.)
 *   ids       T x top int, gates T x top float, contiguous
 *   W1        E * 2I rows of H values: expert e's rows from 2I e on
 *   W2        E * H rows of I values: expert e's rows from H e on
 *   weights   GEMM_MOE_W16: W1 and W2 in `format`, S1 and S2 not read;
 *             GEMM_MOE_MX (gemm_moe.h): MX codes, scales in S1 and S2, pitches in
 *             bytes, T at most GEMM_MOE_MAX_TOKENS and `saved` NULL
 *   Y         T x H in `format`
 *   saved     NULL, or T x top x 2I float for gemm_experts_backward: the rows h
 *             of the choices in an order of their own; rows of dropped choices
 *             are not written
 *   workspace 16-byte aligned, at least gemm_experts_workspace_bytes (else
 *             GEMM_F32_BAD_WORKSPACE); its content is neither read before it
 *             is written nor of use afterwards
 * Sizes outside these bounds: GEMM_F32_INVALID_DIM for negative ones and H or
 * I of 0, else GEMM_F32_BAD_ARG.
 */
int gemm_experts(int T, int E, int top, int H, int I, const void *X, int ldx, const int *ids,
                 const float *gates, int format, const void *W1, int ld1, const unsigned char *S1,
                 int lds1, const void *W2, int ld2, const unsigned char *S2, int lds2, int weights,
                 void *Y, int ldy, float *saved, void *workspace, long long workspace_bytes,
                 void *stream);

/*
 * gemm_experts_backward -- from dY (T x H) the gradients dX (T x H), dgates
 * (T x top float), dW1 and dW2 (rows like W1's and W2's), all in `format` but
 * dgates; for 16-bit weights.  `saved` is what gemm_experts kept for the same X,
 * ids and W1.  Any of the four may be NULL, and is then not computed.  Every
 * element of the others is written: dW1 and dW2 are zeros for experts that no
 * token asks (also where T is 0).
 */
int gemm_experts_backward(int T, int E, int top, int H, int I, const void *dY, int lddy,
                          const void *X, int ldx, const int *ids, const float *gates, int format,
                          const void *W1, int ld1, const void *W2, int ld2, const float *saved,
                          void *dX, int lddx, float *dgates, void *dW1, int lddw1, void *dW2,
                          int lddw2, void *workspace, long long workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_EXPERTS_H */
