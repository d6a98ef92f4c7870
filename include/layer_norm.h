/*
 * layer_norm.h -- C ABI of libcfc_amd, fourth part: the layer norm of rows, with
 * the addition of a residual stream, and its gradients, for AMD Instinct MI355X
 * (gfx950).
 *
 *   h    = x + residual, rounded to the residual's type   (h = x without one)
 *   mean, rstd = 1 / sqrt(mean((h - mean)^2) + eps)       (a row's)
 *   y    = (h - mean) * rstd * weight + bias
 *
 * The conventions of rms_norm.h hold.  Arithmetic and a row's sums are those of
 * 32-bit floats, the variance from differences to the mean.  The weight's and the
 * bias's gradients are summed in a fixed order, in 64 bits over a group of rows (beyond
 * 8192 columns in 32 bits over at most 16 rows); each group's sum is rounded to 32 bits,
 * and those are summed in 64.
 */
#ifndef LAYER_NORM_AMD_H
#define LAYER_NORM_AMD_H

#include <hip/hip_runtime_api.h>

#include "delta_rule.h" /* CFC_TYPE_* */

#ifdef __cplusplus
extern "C" {
#endif

#define LAYER_NORM_MAX_WIDTH 16384

/* x, y [rows, width], weight, bias [width] of `type`; residual, h [rows, width] of
 * `stream_type`, which is `type` or CFC_TYPE_F32; all dense, at any address that
 * their elements' size divides.
 *   residual  NULL: h = x, and h has to be NULL and stream_type = type
 *   h         may be residual itself (or x, where the types are equal), or NULL
 *   bias      or NULL (zeros)
 *   mean, rstd  [rows] float32, or NULL
 *   rows >= 0, 1 <= width <= LAYER_NORM_MAX_WIDTH; eps finite and >= 0 */
int layer_norm_forward(int type, int stream_type, long long rows, long long width, const void *x,
                       const void *residual, const void *weight, const void *bias, float eps, void *y,
                       void *h, float *mean, float *rstd, hipStream_t stream);

/* Bytes of device workspace (16-byte aligned) of layer_norm_backward; -1 for
 * sizes that it refuses. */
long long layer_norm_backward_workspace(long long rows, long long width);

/* With n = (h - mean) * rstd and d = grad_y * weight, means over a row:
 *   grad_x      = rstd * (d - mean(d) - n * mean(d * n)) + grad_h    the gradient
 *                 of h, and so of x and of residual alike
 *   grad_weight = sum over rows of grad_y * n,  grad_bias = sum of grad_y
 *   grad_y [rows, width], weight of `type`; h, grad_h, grad_x of `stream_type`
 *   grad_h      the gradient that h itself has (the residual stream's), or NULL;
 *               grad_x may be grad_h itself
 *   grad_weight, grad_bias  [width] float32, overwritten, zeros for no rows;
 *               grad_bias may be NULL (not wanted) */
int layer_norm_backward(int type, int stream_type, long long rows, long long width, const void *grad_y,
                        const void *h, const void *weight, const float *mean, const float *rstd,
                        const void *grad_h, void *grad_x, float *grad_weight, float *grad_bias,
                        void *workspace, long long workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYER_NORM_AMD_H */
