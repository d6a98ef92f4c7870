/*
 * selective_scan.h -- C ABI of libcfc_amd, seventh part: the selective scan, a recurrent
 * cell whose channels have a state of their own each and decay it by what the input asks
 * for, for AMD Instinct MI355X (gfx950).
 *
 * Per channel the state is h [state]; token t does
 *
 *   D_t = softplus(dt_t + dt_bias)                        (or dt_t + dt_bias)
 *   h_t = exp(D_t a) h_{t-1} + D_t x_t b_t                (a [state] per channel)
 *   y_t = (sum_n c_t h_t + d x_t) z_t sigmoid(z_t)        (without z: no gate)
 *
 * and channel k reads b and c of group k / (channels / groups).
 *
 *   selective_scan_forward    x, dt, a, b, c, d, z, dt_bias, h_0  ->  y, h_T   (sequences)
 *   selective_scan_backward   the gradients of all nine
 *   selective_scan_step       one token for each row of a batch, states in a pool
 *
 * The conventions of delta_rule.h hold: device memory owned by the caller, nothing
 * allocated, synchronised or copied to the host, kernels only enqueued on `stream`
 * (capturable), argument errors (CFC_* codes of cfc.h) before anything is enqueued, no
 * atomics and fixed summation orders, so equal inputs give equal bits.  Arithmetic and
 * states are those of 32-bit floats.  The gradients of a, d and dt_bias are summed in 32 bits
 * over the 4 or 8 tokens of a wave and in 64 over those; what a workgroup has of them is rounded
 * to 32 bits and summed in 64 again.  The decays of up to 8 tokens in a row are multiplied with each
 * other before they meet a state (or its gradient): where states grow so much that this product
 * passes 32 bits, one that is not zero becomes infinite.
 */
#ifndef SELECTIVE_SCAN_AMD_H
#define SELECTIVE_SCAN_AMD_H

#include <hip/hip_runtime_api.h>

#include "delta_rule.h" /* CFC_TYPE_* */

#ifdef __cplusplus
extern "C" {
#endif

/* Compiled limit. */
#define SELECTIVE_SCAN_MAX_STATE 64

/* Bits of clear_rest. */
#define SELECTIVE_SCAN_CLEAR_Y 1
#define SELECTIVE_SCAN_CLEAR_GRAD_X 1
#define SELECTIVE_SCAN_CLEAR_GRAD_DT 2
#define SELECTIVE_SCAN_CLEAR_GRAD_B 4
#define SELECTIVE_SCAN_CLEAR_GRAD_C 8
#define SELECTIVE_SCAN_CLEAR_GRAD_Z 16

/* What the calls share.  Tokens are rows, as in short_conv.h: with `offsets` NULL,
 * sequence s has rows s * seq_len ... (s + 1) * seq_len - 1 (and n_tokens = n_seq *
 * seq_len); otherwise `offsets` is a DEVICE array of n_seq + 1 ints, not decreasing, from
 * 0 to at most n_tokens, and sequence s has rows offsets[s] ... offsets[s + 1] - 1.
 * Sequences of no rows are allowed: their final state is their initial one.  Offsets are
 * not checked on the host; ones that break the rule give undefined outputs, within the
 * arrays' bounds.
 *   x, dt, z, grad_y [n_tokens, channels]: row r at r * stride elements (>= 0), the last
 * axis dense.  b, c [n_tokens, groups, state]: row r, group g at r * stride_t + g *
 * stride_g, the last axis dense; 64 rows of each are less than 2^31 bytes from the first to
 * the last, except for sequences of one row and for a step.  a [channels, state], d, dt_bias [channels] float32,
 * dense, a finite.  States [n_seq, channels, state] float32, dense. */
typedef struct selective_scan_shape {
    int type;           /* CFC_TYPE_* of x, dt, z, b, c, y and their gradients */
    int n_seq;          /* >= 0 */
    int seq_len;        /* read where offsets is NULL */
    long long n_tokens; /* at most 2^31 - 2^16 */
    const int *offsets;
    int channels, groups; /* channels a multiple of groups */
    int state;            /* 1 ... SELECTIVE_SCAN_MAX_STATE */
    int softplus;         /* 1, or 0: D = dt + dt_bias */
    int clear_rest;       /* SELECTIVE_SCAN_CLEAR_*: outputs whose rows behind the last packed sequence become
                             zeros; the others' are left as they were, and all with n_seq = 0 */
    long long x_stride, dt_stride, z_stride, grad_y_stride;
    long long b_stride_t, b_stride_g, c_stride_t, c_stride_g;
} selective_scan_shape_t;

/* y [n_tokens, channels], dense, and final_state (NULL: not wanted) of every sequence,
 * from initial_state (NULL: zeros), which final_state may be.  d NULL: zeros; z NULL: no
 * gate; dt_bias NULL: zeros. */
int selective_scan_forward(const selective_scan_shape_t *shape, const void *x, const void *dt, const float *a,
                           const void *b, const void *c, const float *d, const void *z, const float *dt_bias,
                           const float *initial_state, void *y, float *final_state, hipStream_t stream);

/* Bytes of device workspace (16-byte aligned) of the backward; -1 for a shape that it
 * refuses. */
long long selective_scan_backward_workspace(const selective_scan_shape_t *shape);

/* Gradients of sum(y * grad_y) + sum(final_state * grad_final_state): the forward is
 * recomputed from its inputs, nothing of it is kept.
 *   grad_final_state   or NULL (zeros)
 *   grad_x, grad_dt, grad_z (NULL without z)  [n_tokens, channels], dense
 *   grad_b, grad_c     [n_tokens, groups, state], dense; channels of a group add up
 *   grad_a [channels, state], grad_d, grad_dt_bias [channels] float32, overwritten; the
 *                      last two may be NULL (not wanted)
 *   grad_initial_state or NULL (not wanted); may be grad_final_state itself
 * The workspace's contents on entry are ignored and on return unspecified; it must not
 * overlap any other argument, and calls that may run at the same time need one each. */
int selective_scan_backward(const selective_scan_shape_t *shape, const void *x, const void *dt, const float *a,
                            const void *b, const void *c, const float *d, const void *z, const float *dt_bias,
                            const float *initial_state, const void *grad_y, const float *grad_final_state,
                            void *grad_x, void *grad_dt, float *grad_a, void *grad_b, void *grad_c, float *grad_d,
                            void *grad_z, float *grad_dt_bias, float *grad_initial_state, void *workspace,
                            long long workspace_bytes, hipStream_t stream);

/* One token for each of shape->n_tokens rows; n_seq, seq_len and offsets are not read.
 *   states   [pool, channels, state] float32, updated where they are
 *   slots    DEVICE array of n_tokens ints or NULL: row r's state is states[slots[r]]
 *            (NULL: states[r], pool >= n_tokens).  A slot below 0 or not below `pool`
 *            makes the row idle: its y is zeros and no state changes.  Rows that name
 *            the same slot are taken one after the other in the order of the rows. */
int selective_scan_step(const selective_scan_shape_t *shape, const void *x, const void *dt, const float *a,
                        const void *b, const void *c, const float *d, const void *z, const float *dt_bias,
                        float *states, int pool, const int *slots, void *y, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SELECTIVE_SCAN_AMD_H */
