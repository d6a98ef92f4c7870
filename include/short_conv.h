/*
 * short_conv.h -- C ABI of libcfc_amd, fifth part: the short causal convolution of
 * each channel over a sequence's tokens, in front of the recurrent cells with a large
 * state (delta_rule.h, selective_scan.h), for AMD Instinct MI355X (gfx950).
 *
 *   p_t = bias + sum_{j < width} weight[:, j] x_{t - width + 1 + j}
 *   y_t = p_t sigmoid(p_t), or p_t
 *
 * per channel, where tokens before a sequence's first are its initial state: the
 * width - 1 inputs before it, the oldest first.
 *
 *   short_conv_forward    x, weight, bias, initial state  ->  y, final state
 *   short_conv_backward   the gradients of all four
 *   short_conv_step       one token for each row of a batch, states in a pool
 *
 * The conventions of delta_rule.h hold: device memory owned by the caller, nothing
 * allocated, synchronised or copied to the host, kernels only enqueued on `stream`
 * (capturable), argument errors (CFC_* codes of cfc.h) before anything is enqueued, no
 * atomics and fixed summation orders, so equal inputs give equal bits.  Arithmetic is
 * that of 32-bit floats; the weight's and the bias's gradients are summed in 64 bits over
 * groups of 16 or 32 tokens.
 */
#ifndef SHORT_CONV_AMD_H
#define SHORT_CONV_AMD_H

#include <hip/hip_runtime_api.h>

#include "delta_rule.h" /* CFC_TYPE_* */

#ifdef __cplusplus
extern "C" {
#endif

/* Compiled limits: widths of 2, 3 and 4. */
#define SHORT_CONV_MAX_WIDTH 4

/* What the calls share.  Tokens are rows: with `offsets` NULL, sequence s has rows
 * s * seq_len ... (s + 1) * seq_len - 1 (and n_tokens = n_seq * seq_len); otherwise
 * `offsets` is a DEVICE array of n_seq + 1 ints, not decreasing, from 0 to at most
 * n_tokens, and sequence s has rows offsets[s] ... offsets[s + 1] - 1.  Sequences of no
 * rows are allowed.  Offsets are not checked on the host; ones that break the rule give undefined outputs,
 * within the arrays' bounds.
 *   x [n_tokens, channels]: row r at r * x_stride elements (>= 0), so that a slice of a
 * projection can be read where it lies, the last axis dense; grad_y likewise.  weight
 * [channels, width], bias [channels] and the states [n_seq, width - 1, channels] of the
 * same type, dense. */
typedef struct short_conv_shape {
    int type;           /* CFC_TYPE_* of all tensors but the weights' gradients */
    int n_seq;          /* >= 0 */
    int seq_len;        /* read where offsets is NULL */
    long long n_tokens; /* at most 2^31 - 2^16 */
    const int *offsets;
    int channels; /* >= 1 */
    int width;    /* 2, 3 or 4 */
    int silu;     /* 1: y = p sigmoid(p); 0: y = p */
    int clear_rest; /* rows of y and grad_x behind the last packed sequence: 1 makes them zeros, 0 leaves them
                       (as n_seq = 0 does) */
    long long x_stride, grad_y_stride;
} short_conv_shape_t;

/* y [n_tokens, channels], dense.  bias NULL: zeros; initial_state NULL: zeros;
 * final_state (the last width - 1 inputs of each sequence, from its initial state where
 * it is shorter) NULL: not wanted; it may be initial_state itself. */
int short_conv_forward(const short_conv_shape_t *shape, const void *x, const void *weight, const void *bias,
                       const void *initial_state, void *y, void *final_state, hipStream_t stream);

/* Bytes of device workspace (16-byte aligned) of the backward; -1 for a shape that it
 * refuses. */
long long short_conv_backward_workspace(const short_conv_shape_t *shape);

/* Gradients of sum(y * grad_y) + sum(final_state * grad_final_state).
 *   grad_final_state    or NULL (zeros)
 *   grad_x              [n_tokens, channels], dense
 *   grad_weight         [channels, width] float32, overwritten
 *   grad_bias           [channels] float32, or NULL (not wanted)
 *   grad_initial_state  the states' type, or NULL (not wanted) */
int short_conv_backward(const short_conv_shape_t *shape, const void *x, const void *weight, const void *bias,
                        const void *initial_state, const void *grad_y, const void *grad_final_state,
                        void *grad_x, float *grad_weight, float *grad_bias, void *grad_initial_state,
                        void *workspace, long long workspace_bytes, hipStream_t stream);

/* One token for each of shape->n_tokens rows; n_seq, seq_len and offsets are not read.
 *   states   [pool, width - 1, channels], updated where they are
 *   slots    DEVICE array of n_tokens ints or NULL: row b's state is states[slots[b]]
 *            (NULL: states[b], pool >= n_tokens).  A slot below 0 or not below `pool`
 *            makes the row idle: its y is zeros and no state changes.  Rows that name
 *            the same slot are taken one after the other in the order of the rows. */
int short_conv_step(const short_conv_shape_t *shape, const void *x, const void *weight, const void *bias,
                    void *states, int pool, const int *slots, void *y, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SHORT_CONV_AMD_H */
