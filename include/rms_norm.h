/*
 * rms_norm.h -- C ABI of libcfc_amd, third part: the root-mean-square norm of
 * rows, with the addition of a residual stream and an output in 8 bits, for AMD
 * Instinct MI355X (gfx950).
 *
 *   h    = x + residual, rounded to the residual's type   (h = x without one)
 *   rstd = 1 / sqrt(mean(h^2) + eps)                      (a row's)
 *   y    = h * rstd * weight
 *
 *   rms_norm_forward        y in x's type
 *   rms_norm_forward_e4m3   y in e4m3 with scales: y ~ e4m3 value * scale
 *   rms_norm_backward       the gradients of h and weight
 *
 * The conventions of cfc.h hold: device memory owned by the caller, nothing
 * allocated, synchronised or copied to the host, kernels only enqueued on
 * `stream` (capturable), argument errors before anything is enqueued, no atomics
 * and fixed summation orders, 64-bit offsets.  Arithmetic and sums are those of
 * 32-bit floats; the weight gradient's terms are summed in 64 bits.  The norm is
 * that of the rounded h, so that the backward, which reads the rounded h, is the
 * gradient of what the forward computed.
 */
#ifndef RMS_NORM_AMD_H
#define RMS_NORM_AMD_H

#include <hip/hip_runtime_api.h>

#include "delta_rule.h" /* CFC_TYPE_* */

#ifdef __cplusplus
extern "C" {
#endif

#define RMS_NORM_MAX_WIDTH 16384

/* x, y [rows, width] and weight [width] of `type`; residual, h [rows, width] of
 * `stream_type`, which is `type` or CFC_TYPE_F32; all dense.
 *   residual  NULL: h = x, and h has to be NULL and stream_type = type
 *   h         may be residual itself (or x, where the types are equal), or NULL
 *   rstd      [rows] float32, or NULL
 *   rows >= 0, 1 <= width <= RMS_NORM_MAX_WIDTH; eps finite and >= 0 */
int rms_norm_forward(int type, int stream_type, long long rows, long long width, const void *x,
                     const void *residual, const void *weight, float eps, void *y, void *h,
                     float *rstd, hipStream_t stream);

/* y in e4m3 (finite values to 448, round to nearest even), y ~ value * scale.
 *   group   columns that share a scale: 0 for a whole row, or a power of two
 *           from 16 to 512 (the last group of a row may be shorter)
 *   y       [rows, width] bytes
 *   scales  [rows, ceil(width / group)] float32: the group's largest |y| / 448,
 *           or 1 / 448 where all are zero
 * The rest is rms_norm_forward's. */
int rms_norm_forward_e4m3(int type, int stream_type, long long rows, long long width, const void *x,
                          const void *residual, const void *weight, float eps, int group, void *y,
                          float *scales, void *h, float *rstd, hipStream_t stream);

/* Bytes of device workspace (16-byte aligned) of rms_norm_backward; -1 for sizes
 * that it refuses. */
long long rms_norm_backward_workspace(long long rows, long long width);

/* With n = h * rstd and d = grad_y * weight:
 *   grad_x      = rstd * (d - n * mean(d * n)) + grad_h    the gradient of h,
 *                 and so of x and of residual alike
 *   grad_weight = sum over rows of grad_y * n
 *   grad_y [rows, width], weight of `type`; h, grad_h, grad_x of `stream_type`
 *   grad_h      the gradient that h itself has (the residual stream's), or NULL;
 *               grad_x may be grad_h itself
 *   grad_weight [width] float32, overwritten; zeros for no rows */
int rms_norm_backward(int type, int stream_type, long long rows, long long width, const void *grad_y,
                      const void *h, const void *weight, const float *rstd, const void *grad_h,
                      void *grad_x, float *grad_weight, void *workspace, long long workspace_bytes,
                      hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RMS_NORM_AMD_H */
