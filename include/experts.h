/*
 * experts.h -- C ABI of the tokens' way to their experts and back
 * (libsgemm_f32.so): a router's choice, the stable sort of the choices by expert, the
 * copy of the token rows into that order, the weighted sum of the experts'
 * rows per token, and the gradients.
 *
 * T tokens choose J experts each (J choices per token, in order).  A choice
 * outside 0 .. E-1 is dropped.  The R = T*J places hold the choices that are
 * not dropped, sorted by expert and in each expert by (token, choice):
 *     rows[t*J + j]  the place of choice j of token t, or -1
 *     offsets[e]     the first place of expert e; offsets[E] = places in use
 *
 * Conventions are those of sgemm_f32.h (checks on the host, asynchronous,
 * nothing allocated, sgemm_status codes); types are linear_type.  Sums over
 * a token's choices are in FP32 in the order of the choices, rounded once.
 * Nothing depends on the order in which threads run.
 */
#ifndef EXPERTS_H
#define EXPERTS_H

#include "linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most choices per token. */
#define EXPERTS_MAX_CHOICES 64
/* Most experts and groups of expert_choose. */
#define EXPERTS_MAX_CHOOSE 1024
#define EXPERTS_MAX_GROUPS 32

typedef enum { EXPERTS_SOFTMAX = 0, EXPERTS_SIGMOID = 1 } experts_scoring;

/*
 * expert_choose -- each token's J experts and their weights from a router's logits l.
 *     s = softmax(l) or 1 / (1 + exp(-l)),  v = s + bias
 * The E experts form `groups` equal groups in a row; those kept_groups compete
 * whose group_top (1 or 2) best v have the largest sum.  Of their experts the J
 * with the largest v are chosen, in falling order; of equal values the lowest
 * number comes first, for groups as for experts.  Without a bias the order is
 * that of the logits (and that of a group its best logit, if group_top is 1);
 * else it is that of v computed in 64 bits.
 *     weights[t*J + j] = scale * s, or scale * s / sum of the chosen s (renormalize)
 * The bias decides the choice and enters no weight.
 *   logits, ldl : T x E of `type`, ldl >= E.
 *   bias        : E FP32 values, or NULL.
 *   chosen      : T*J 32-bit values (out).     weights : T*J FP32 values (out).
 * An expert with a logit or a bias of minus infinity (or a bias that is no
 * number) is never chosen.  Places for which no expert is left have chosen -1,
 * which expert_sort drops, and weight 0: a token whose logits are all minus
 * infinity goes to no expert.  A token with a NaN among its logits, or with
 * softmax plus infinity, chooses none, and its weights are NaN.
 * E is at most EXPERTS_MAX_CHOOSE, J at most EXPERTS_MAX_CHOICES and E, groups
 * at most EXPERTS_MAX_GROUPS and a divisor of E.
 */
int expert_choose(int type, int T, int E, int J, const void *logits, int64_t ldl, const float *bias, int scoring,
                  int groups, int kept_groups, int group_top, int renormalize, float scale, int *chosen,
                  float *weights, cudaStream_t stream);

/*
 * expert_choose_backward -- the logits' gradient from the weights'.
 *   dweights, chosen : T*J values; a choice outside 0 .. E-1 counts for nothing.
 *   dlogits, ldd     : T x E of `type`, written whole: 0 for experts that the
 *                      weights do not depend on.
 */
int expert_choose_backward(int type, int T, int E, int J, const float *dweights, const int *chosen,
                           const void *logits, int64_t ldl, int scoring, int renormalize, float scale,
                           void *dlogits, int64_t ldd, cudaStream_t stream);

/*
 * expert_sort -- rows and offsets from the choices.
 *   choices      : T*J experts, 32-bit (choice_bytes 4) or 64-bit (8) signed.
 *   rows         : T*J 32-bit values (out).
 *   offsets      : E+1 32-bit values (out).
 *   workspace    : expert_sort_workspace_size(T, J, E) bytes, 16-byte aligned
 *                  (NULL where that is 0).
 * T*J is at most 2^31 - 1; E 1 .. LINEAR_MAX_EXPERTS.  T == 0 or J == 0 still
 * writes the offsets (all 0).
 */
int expert_sort(int T, int J, int E, const void *choices, int choice_bytes,
                int *rows, int *offsets,
                void *workspace, size_t workspace_bytes, cudaStream_t stream);
size_t expert_sort_workspace_size(int T, int J, int E);

/*
 * expert_gather -- xs[rows[t*J + j]] = x[t]; the places from offsets[E] on
 * are set to 0.
 *   x, ldx   : T x H.     xs, ldxs : T*J x H.
 */
int expert_gather(int type, int T, int J, int H, int E, const int *rows, const int *offsets,
                  const void *x, int64_t ldx, void *xs, int64_t ldxs, cudaStream_t stream);

/*
 * expert_combine -- y[t] = residual[t] + sum_j weights[t*J + j] ys[rows[t*J + j]].
 *   weights  : T*J FP32 values, or NULL (all 1: the gradient of expert_gather).
 *   ys, ldys : T*J x H.   residual, ldr : T x H or NULL (may be y itself).
 *   y, ldy   : T x H.  A token without a place gives residual[t], or 0.
 */
int expert_combine(int type, int T, int J, int H, const int *rows, const float *weights,
                   const void *ys, int64_t ldys, const void *residual, int64_t ldr,
                   void *y, int64_t ldy, cudaStream_t stream);

/*
 * expert_combine_backward -- dys[rows[t*J + j]] = weights[t*J + j] dy[t] (0 in
 * the places from offsets[E] on) and dweights[t*J + j] = dy[t] . ys[rows[t*J + j]]
 * (0 for a dropped choice).
 *   dys, lddys : T*J x H.   dweights : T*J FP32 values, or NULL (then ys may
 *   be NULL).  weights may be NULL (all 1).
 */
int expert_combine_backward(int type, int T, int J, int H, int E, const int *rows, const int *offsets,
                            const float *weights, const void *dy, int64_t lddy, const void *ys, int64_t ldys,
                            void *dys, int64_t lddys, float *dweights, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EXPERTS_H */
