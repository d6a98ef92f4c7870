/*
 * grad_norm.h -- C ABI of libcfc_amd, sixth part: the norm of all gradients of a model
 * together, and clipping to it, for AMD Instinct MI355X (gfx950).
 *
 *   norm = sqrt(sum over all tensors of g^2)
 *   out  = g * min(1, max_norm / (norm + 1e-6))
 *
 * The conventions of cfc.h hold: device memory owned by the caller, nothing allocated,
 * synchronised or copied to the host (the factor stays on the GPU), kernels only enqueued
 * on `stream` (capturable), argument errors before anything is enqueued, no atomics and
 * fixed summation orders, so equal inputs give equal bits.  Squares are summed in 64 bits,
 * so that no square of a finite gradient overflows; a clipped gradient is a product of
 * 32-bit floats, rounded once to its type.
 */
#ifndef GRAD_NORM_AMD_H
#define GRAD_NORM_AMD_H

#include <hip/hip_runtime_api.h>

#include "delta_rule.h" /* CFC_TYPE_* */

#ifdef __cplusplus
extern "C" {
#endif

/* A tensor of `numel` elements (>= 0) of a CFC_TYPE_*, dense.  `out`, read by
 * clip_grad_norm alone, gets as many of the same type; it may be `grad` itself. */
typedef struct grad_tensor {
    const void *grad;
    void *out;
    long long numel;
    int type;
} grad_tensor_t;

/* Bytes of device workspace (16-byte aligned) of the calls below for so many tensors,
 * whatever their sizes; -1 for a negative count. */
long long grad_norm_workspace(int count);

/* norm [1] of `count` tensors; 0 for none.  `tensors` is a HOST array, read before the
 * call returns.  A tensor may be named twice and counts twice.  NaN where any element is,
 * infinite where one is infinite or the norm passes 32 bits. */
int grad_norm(const grad_tensor_t *tensors, int count, float *norm, void *workspace, long long workspace_bytes,
              hipStream_t stream);

/* norm [1] as above, of the gradients as they were given, and every tensor's `out`.
 *   max_norm  >= 0, or infinite: nothing is clipped
 * Outputs must not overlap each other, nor any gradient but their own.  Where the norm is
 * NaN all outputs are; where it is infinite, that of finite gradients past 32 bits too, the
 * factor is 0, and with an infinite max_norm 1. */
int clip_grad_norm(const grad_tensor_t *tensors, int count, float max_norm, float *norm, void *workspace,
                   long long workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GRAD_NORM_AMD_H */
