/*
 * gemm_route.h -- C ABI of the routing of tokens to experts of the gemm_f32
 * library (MI355X, gfx950): scores, the choice of experts and their gates, and
 * the gradient of the logits.  The experts' products are in gemm_experts.h.
 *
 * For each of T tokens (rows z of Z):
 *   s[e]    = exp(z[e]) / sum over all E of exp(z)   (GEMM_ROUTE_SOFTMAX), or
 *             1 / (1 + exp(-z[e]))                   (GEMM_ROUTE_SIGMOID)
 *   key[e]  = s[e] + bias[e]; the bias decides the choice, and is in no gate
 *   The experts are `groups` runs of E / groups.  Where top_groups < groups, a
 *   group's score is the largest key in it (GEMM_ROUTE_MAX) or the sum of its
 *   two largest (GEMM_ROUTE_TOP2; of one if it has one), and only experts of the
 *   top_groups groups of largest score can be chosen.
 *   chosen  = the `top` experts of largest key, in falling order
 *   gate[s] = scale s[chosen s], or, with `renormalize`, over the sum of s[chosen]
 * Of equal keys or scores the lower index comes first.  Without a bias experts
 * (and groups, by GEMM_ROUTE_MAX) are ordered by their logits, which is the same
 * order, also where s is rounded to 0 or 1.  Everything is computed in 64 bits;
 * each gate is rounded once.
 *
 * An expert whose logit is -infinity (masked) or NaN, or whose key is, comes after
 * all others of its groups; a group of such alone comes after all other groups.
 * A masked expert's gate is 0, and so are all of a token whose chosen experts'
 * scores are all 0.  A logit of +infinity is the limit: it and its equals share
 * the softmax.  A NaN makes NaN the gates whose sum it enters.
 *
 * Memory, streams and errors are as for gemm_f32 (gemm_f32.h): device
 * pointers owned by the caller, nothing allocated, asynchronous on `stream`,
 * argument errors returned before anything is enqueued, status codes
 * GEMM_F32_*.  Outputs must not overlap inputs or one another.
 */
#ifndef GEMM_ROUTE_H
#define GEMM_ROUTE_H

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_ROUTE_SOFTMAX 0
#define GEMM_ROUTE_SIGMOID 1
#define GEMM_ROUTE_MAX 0
#define GEMM_ROUTE_TOP2 1

#define GEMM_ROUTE_MAX_TOKENS (1 << 22)
#define GEMM_ROUTE_MAX_EXPERTS 512
#define GEMM_ROUTE_MAX_TOP 16
#define GEMM_ROUTE_MAX_GROUPS 64

/*
 * gemm_moe_route
 *   T           0 .. GEMM_ROUTE_MAX_TOKENS (0: no-op)
 *   E, top      1 <= top <= E; at most GEMM_ROUTE_MAX_EXPERTS, GEMM_ROUTE_MAX_TOP
 *   Z           T x E in `format` (GEMM_MIXED_BF16, GEMM_MIXED_F16 or
 *               GEMM_MX_F32), element-aligned, pitch ldz in elements
 *   bias        E float, or NULL
 *   groups      1 .. GEMM_ROUTE_MAX_GROUPS, E a multiple of it
 *   top_groups  1 .. groups; top <= top_groups * E / groups
 *   scale       finite
 *   ids, gates  T x top int and float, contiguous, 4-byte aligned
 * Sizes outside these bounds: GEMM_F32_INVALID_DIM for negative ones, else
 * GEMM_F32_BAD_ARG.
 */
int gemm_moe_route(int T, int E, int top, const void *Z, int ldz, int format, int score,
                   const float *bias, int groups, int top_groups, int group_score,
                   int renormalize, float scale, int *ids, float *gates, void *stream);

/*
 * gemm_moe_route_backward -- dZ, the gradient of the logits (T x E in `format`,
 * pitch lddz) from that of the gates (T x top float, contiguous), for the chosen
 * experts `ids` that gemm_moe_route gave for the same Z, score, renormalize and
 * scale.  Every element of dZ is written; the choice has no gradient.  An id
 * outside 0 .. E - 1 adds nothing.
 */
int gemm_moe_route_backward(int T, int E, int top, const float *dgates, const void *Z, int ldz,
                            int format, int score, int renormalize, float scale, const int *ids,
                            void *dZ, int lddz, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_ROUTE_H */
