/*
 * delta_rule.h -- C ABI of libcfc_amd, second part: the gated delta rule, a
 * recurrent cell with a matrix state, for AMD Instinct MI355X (gfx950).
 *
 * Per value head the state is S [dim_k, dim_v]; token t does
 *
 *   S'  = exp(g_t) S_{t-1}                     (decay)
 *   u_t = beta_t (v_t - S'^T k_t)              (what the state gets wrong for k_t)
 *   S_t = S' + k_t u_t^T
 *   o_t = scale * S_t^T q_t
 *
 * and value head h reads query and key head h / (heads_v / heads_k).
 *
 *   delta_rule_forward    q, k, v, g, beta, S_0  ->  o, S_T       (sequences)
 *   delta_rule_backward   the gradients of q, k, v, g, beta, S_0
 *   delta_rule_step       one token for each row of a batch, states in a pool
 *
 * The conventions of cfc.h hold: device memory owned by the caller, nothing
 * allocated, synchronised or copied to the host, kernels only enqueued on
 * `stream` (capturable), argument errors (CFC_* codes of cfc.h) before anything
 * is enqueued, no atomics and fixed summation orders, so equal inputs give
 * equal bits.  Different from cfc.h: the tensors' type is an argument and the
 * arithmetic is that of 32-bit floats (decays are summed in 64 bits).
 */
#ifndef DELTA_RULE_AMD_H
#define DELTA_RULE_AMD_H

#include <hip/hip_runtime_api.h>

#include "cfc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of q, k, v, o and their gradients. */
#define CFC_TYPE_F32 0
#define CFC_TYPE_BF16 1
#define CFC_TYPE_F16 2

/* Compiled limits. */
#define DELTA_MAX_DIM_K 128
#define DELTA_MAX_DIM_V 256

/* What the sequence calls share.  Tokens are rows: with `offsets` NULL, sequence
 * s has rows s * seq_len ... (s + 1) * seq_len - 1 (and n_tokens = n_seq *
 * seq_len); otherwise `offsets` is a DEVICE array of n_seq + 1 ints, not
 * decreasing, from 0 to at most n_tokens, and sequence s has rows offsets[s] ...
 * offsets[s + 1] - 1.  Sequences of no rows are allowed: their final state is
 * their initial one.  Output rows behind the last sequence are left as they were.
 * Offsets are not checked on the host; ones that break the rule give undefined
 * outputs, within the arrays' bounds.  Packed sequences are taken in groups of 64
 * tokens unless they have 8 to 32 in all: single tokens of many belong in
 * delta_rule_step.
 *   q, k [n_tokens, heads_k, dim_k], v [n_tokens, heads_v, dim_v]: row r, head h
 * at r * stride_t + h * stride_h elements (strides >= 0, so a slice of a fused
 * projection or a broadcast head can be read where it lies), the last axis
 * dense; 64 rows are less than 2^31 bytes (except for a step, a forward of sequences
 * so short that it takes no workspace, and sequences of one row).  g, beta
 * [n_tokens, heads_v] float32, dense: the decay's logarithm (-inf: forget all)
 * and the gate.  States [n_seq, heads_v, dim_k, dim_v] float32, dense. */
typedef struct delta_rule_shape {
    int type;             /* CFC_TYPE_* of q, k, v, o, grad_o, grad_q, grad_k, grad_v */
    int n_seq;            /* >= 0 */
    int seq_len;          /* read where offsets is NULL */
    long long n_tokens;   /* < 2^31; for the sequences' calls at most 2^23 groups of 64 */
    const int *offsets;
    int heads_k, heads_v; /* heads_v a multiple of heads_k */
    int dim_k, dim_v;     /* 1 ... DELTA_MAX_DIM_K, 1 ... DELTA_MAX_DIM_V */
    float scale;          /* of o; finite */
    long long q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h;
    long long go_stride_t, go_stride_h; /* of grad_o, read by the backward */
} delta_rule_shape_t;

/* Bytes of device workspace (16-byte aligned) of the two calls below; -1 for a
 * shape they refuse.  0 where none is needed.  It grows with the groups of 64 tokens
 * (packed, n_tokens / 64 + n_seq of them): with dims of 128 in bf16 and two value heads a
 * key head, 75 KB a group and value head for the forward, 305 KB for the gradients (8192
 * tokens of 32 heads 307 MB and 1.25 GB). */
long long delta_rule_forward_workspace(const delta_rule_shape_t *shape);
long long delta_rule_backward_workspace(const delta_rule_shape_t *shape);

/* o [n_tokens, heads_v, dim_v] and final_state (NULL: not wanted) of every
 * sequence, from initial_state (NULL: zeros).  final_state may be initial_state
 * itself.  The workspace's contents on entry are ignored and on return
 * unspecified; it must not overlap any other argument, and calls that may run
 * at the same time need one each.
 * A value that is not finite in q, k, v, g or beta makes the outputs of its own
 * sequence undefined from the beginning of its group of 64 tokens on, and all
 * gradients of that sequence; so does a 32-bit one that rounds to infinity in bf16
 * (from 2^128 - 2^119 on). */
int delta_rule_forward(const delta_rule_shape_t *shape, const void *q, const void *k, const void *v,
                       const float *g, const float *beta, const float *initial_state, void *o,
                       float *final_state, void *workspace, long long workspace_bytes,
                       hipStream_t stream);

/* Gradients of sum(o * grad_o) + sum(final_state * grad_final_state): the
 * forward is recomputed from its inputs, nothing of it is kept.
 *   grad_o            [n_tokens, heads_v, dim_v], strided as shape says
 *   grad_final_state  or NULL (zeros)
 *   grad_q, grad_k, grad_v   dense, the shapes of q, k, v; heads that share a
 *                     query and key head add up in it
 *   grad_g, grad_beta [n_tokens, heads_v] float32
 *   grad_initial_state  or NULL (not wanted); may be grad_final_state itself */
int delta_rule_backward(const delta_rule_shape_t *shape, const void *q, const void *k, const void *v,
                        const float *g, const float *beta, const float *initial_state,
                        const void *grad_o, const float *grad_final_state, void *grad_q, void *grad_k,
                        void *grad_v, float *grad_g, float *grad_beta, float *grad_initial_state,
                        void *workspace, long long workspace_bytes, hipStream_t stream);

/* One token for each of `batch` rows: shape->n_tokens = batch, n_seq, seq_len
 * and offsets are not read; q, k, v, g, beta, o as above with a row for each
 * token.
 *   states   [pool, heads_v, dim_k, dim_v] float32, updated where they are
 *   slots    DEVICE array of `batch` ints or NULL: row b's state is
 *            states[slots[b]] (NULL: states[b], pool >= batch).  A slot below 0
 *            or not below `pool` makes the row idle: its o is zeros and no
 *            state changes.  Rows that name the same slot are taken one after
 *            the other in the order of the rows. */
int delta_rule_step(const delta_rule_shape_t *shape, const void *q, const void *k, const void *v,
                    const float *g, const float *beta, float *states, int pool, const int *slots,
                    void *o, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DELTA_RULE_AMD_H */
