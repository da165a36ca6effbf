/*
 * cross_entropy.h -- C ABI of a head's loss (libsgemm_f32.so): the softmax cross
 * entropy of a matrix product's rows, and its gradient, without the product in
 * memory.
 *
 *     z[i][j] = sum_k x[i][k] w[k][j]
 *     lse[i]  = log sum_j exp(z[i][j])
 *     loss[i] = lse[i] - z[i][targets[i]], or 0 for a target outside 0 .. N-1
 * and, for gradients dloss of loss and dlse of lse (with dloss[i] taken for 0
 * where there is no target):
 *     dz[i][j] = (dloss[i] + dlse[i]) exp(z[i][j] - lse[i]) - dloss[i] [j = targets[i]]
 *     dx = dz.w^T,  dw = x^T.dz
 *
 * x is M x K (tokens), w is K x N (the vocabulary) in either order, as in
 * linear.h; both and the gradients have one type, losses, log sums and their
 * gradients are FP32.  Products are those of linear.h: exact, added in FP32
 * (FP32: six products of bf16 pieces); logits by blocks of K (at most 512 in 16 bits, 64
 * in FP32), whose sums are added with round-to-nearest.  The forward pass keeps two numbers per
 * token and 32 to 128 columns (FP32 up to 64 tokens: the logits, in the workspace); the gradient makes the logits again, some of the
 * vocabulary at a time, and keeps at most CROSS_ENTROPY_PIECE of dz.
 * The 16-bit types round dz to themselves before the two products, as fractions
 * of the largest finite |dloss| and |dloss + dlse| (float16: times 2^14), so that with equal losses the
 * targets' -1 is exact and small gradients do not vanish.
 * Sums have a fixed order: a call gives the same bits every time.
 *
 * Conventions are those of linear.h (checks on the host, asynchronous, nothing
 * allocated, sgemm_status codes, bounded waits that linear_timeouts reports).
 */
#ifndef CROSS_ENTROPY_H
#define CROSS_ENTROPY_H

#include "linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most values of dz at a time (more where 256 columns have more). */
#define CROSS_ENTROPY_PIECE (1 << 28)

/*
 * linear_cross_entropy_forward
 *   targets      : M values, 32-bit (target_bytes 4) or 64-bit (8) signed.
 *   loss, lse    : M FP32 values each (out).
 *   workspace    : DEVICE memory, 256-byte aligned, of
 *                  linear_cross_entropy_forward_workspace_size bytes for the
 *                  same arguments (NULL where that is 0).
 * K == 0 gives log N; N == 0 gives minus infinity for lse.
 */
int linear_cross_entropy_forward(int type, int M, int N, int K, const void *x, int64_t ldx, const void *w, int64_t ldw,
                                 int w_order, const void *targets, int target_bytes, float *loss, float *lse,
                                 void *workspace, size_t workspace_bytes, cudaStream_t stream);
size_t linear_cross_entropy_forward_workspace_size(int type, int M, int N, int K, const void *x, int64_t ldx,
                                                   const void *w, int64_t ldw, int w_order);

/*
 * linear_cross_entropy_backward
 *   dloss, dlse  : M FP32 values; either may be NULL (all 0).
 *   lse          : M FP32 values, as the forward pass gave them.
 *   dx, lddx     : M x K, or NULL (not wanted).
 *   dw, lddw     : like w, in the order of w_order, or NULL.
 */
int linear_cross_entropy_backward(int type, int M, int N, int K, const float *dloss, const float *dlse, const void *x,
                                  int64_t ldx, const void *w, int64_t ldw, int w_order, const void *targets,
                                  int target_bytes, const float *lse, void *dx, int64_t lddx, void *dw, int64_t lddw,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream);
size_t linear_cross_entropy_backward_workspace_size(int type, int M, int N, int K, const void *x, int64_t ldx,
                                                    const void *w, int64_t ldw, int w_order, int want_dx, int want_dw);

#ifdef __cplusplus
}
#endif

#endif /* CROSS_ENTROPY_H */
