/*
 * norm.h -- C ABI of layer norm and its gradient (libsgemm_f32.so).
 *
 *     mean_i = sum_j x[i][j] / N,   rstd_i = 1 / sqrt(sum_j (x[i][j] - mean_i)^2 / N + eps)
 *     h[i][j] = (x[i][j] - mean_i) rstd_i
 *     y[i][j] = h[i][j] weight[j] + bias[j]
 * and, for a gradient dy of y, with g = dy weight:
 *     dx[i][j] = rstd_i (g[i][j] - sum_j g[i][j] / N - h[i][j] sum_j g[i][j] h[i][j] / N)
 *     dweight[j] = sum_i dy[i][j] h[i][j],   dbias[j] = sum_i dy[i][j]
 *
 * All tensors of a call have one type (linear_type), but the statistics, which
 * are FP32.  Everything up to the one rounding of a result is in FP32; the
 * variance is taken from the differences to the mean, and what rounding leaves
 * of the mean is taken off them again, in the gradient too: rows far from zero
 * lose nothing to that.  Sums have a fixed order: a call gives the same bits
 * every time.
 *
 * Conventions are those of sgemm_f32.h: arguments are checked on the host
 * before anything is launched, work is only enqueued on `stream`, nothing is
 * allocated, status codes are sgemm_status.
 */
#ifndef NORM_H
#define NORM_H

#include "linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * layer_norm_forward
 *   x, ldx  : M x N, ldx >= max(1, N) elements between rows.
 *   weight  : N values, or NULL (all 1).     bias : N values, or NULL (all 0).
 *   eps     : >= 0 and finite.
 *   stats   : M x 2 FP32 values (out): mean and rstd of each row, for the
 *             gradient; or NULL.
 *   y, ldy  : M x N.
 * M == 0 is a no-op; N == 0 leaves the statistics at 0.  Nothing written may
 * overlap anything else of the call (SGEMM_ERR_ALIAS).
 */
int layer_norm_forward(int type, int M, int N, const void *x, int64_t ldx, const void *weight, const void *bias,
                       float eps, float *stats, void *y, int64_t ldy, cudaStream_t stream);

/*
 * layer_norm_backward
 *   dy, lddy : M x N.     stats : as layer_norm_forward left them.
 *   dx, lddx : M x N, or NULL (not wanted).
 *   dweight, dbias : N values, or NULL.  M == 0 gives zeros.
 *   workspace : DEVICE memory, 256-byte aligned, of
 *               layer_norm_backward_workspace_size bytes (NULL where that is 0).
 */
int layer_norm_backward(int type, int M, int N, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                        const void *weight, const float *stats, void *dx, int64_t lddx, void *dweight, void *dbias,
                        void *workspace, size_t workspace_bytes, cudaStream_t stream);
size_t layer_norm_backward_workspace_size(int M, int N, int want_dweight, int want_dbias);

#ifdef __cplusplus
}
#endif

#endif /* NORM_H */
