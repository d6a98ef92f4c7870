"""Tensor checks and pointer marshalling of the gated delta rule (include/delta_rule.h)."""
from __future__ import annotations

from ctypes import byref
from typing import Optional, Tuple

import torch

from ._lib import DeltaRuleShape, _check, load_library
from ._tensors import F32, check, element_type, given_or_new, on_device, ptr, space, stream_ptr


def _rows(t, name, lead, dtype, device, shape=None):
    """(token stride, head stride) of t [*lead, heads, dim], rows numbered along its leading axes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dim() != lead + 2 or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a {lead + 2}-dimensional tensor on a GPU, of q's type and device "
                         f"(got {t.dim()} dimensions, {t.dtype}, {t.device})")
    n = t.shape
    if shape is not None and n != shape:
        raise ValueError(f"{name} has shape {tuple(n)}, expected {tuple(shape)}")
    st = t.stride()
    if st[-1] != 1 and n[-1] > 1 and t.numel():
        raise ValueError(f"{name}'s last axis must be dense (its stride is {st[-1]})")
    if lead == 1:
        return st[0], st[1]
    if n[1] == 1:
        return st[0], st[2]
    if st[0] != n[1] * st[1] and n[0] > 1 and t.numel():
        raise ValueError(f"{name}'s sequences must lie one behind the other (strides {st}): make it contiguous")
    return st[1], st[2]


def _ints(*sizes):
    if max(sizes) > 0x7fffffff:  # ctypes would pass their low 32 bits
        raise ValueError(f"sizes {sizes} do not fit 32 bits")


def _shape(q, k, v, g, beta, scale, offsets, lead, grad_o=None):
    kind, dtype, dev, n = element_type(q, "q"), q.dtype, q.device, q.shape
    qs = _rows(q, "q", lead, dtype, dev)
    ks = _rows(k, "k", lead, dtype, dev, n)
    vs = _rows(v, "v", lead, dtype, dev)
    nv = v.shape
    if nv[:lead] != n[:lead]:
        raise ValueError(f"v has shape {tuple(nv)}, expected {tuple(n[:lead])} tokens as q has")
    gs = (0, 0) if grad_o is None else _rows(grad_o, "grad_o", lead, dtype, dev, nv)
    heads_k, dim_k, heads_v, dim_v = n[-2], n[-1], nv[-2], nv[-1]
    if dim_k < 1 or dim_v < 1:
        raise ValueError(f"q and v have heads of {dim_k} and {dim_v} elements, expected at least 1")
    if heads_k < 1 or heads_v < 1 or heads_v % heads_k:
        raise ValueError(f"v's {heads_v} heads are no multiple of q's {heads_k}")
    gates = nv[:-1]
    check(g, "g", F32, dev, gates)
    check(beta, "beta", F32, dev, gates)
    tokens, count, length, at = n[0] if lead == 1 else n[0] * n[1], 0, 0, None
    if offsets is not None:
        check(offsets, "offsets", torch.int32, dev)
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError("offsets must be a vector of the sequences' beginnings and the last one's end")
        count, at = offsets.numel() - 1, offsets.data_ptr()
    elif lead == 2:
        count, length = n[0], n[1]
    _ints(count, length, heads_v, dim_k, dim_v)
    return DeltaRuleShape(kind, count, length, tokens, at, heads_k, heads_v, dim_k, dim_v,
                          dim_k ** -0.5 if scale is None else scale, *qs, *ks, *vs, *gs)


def _lead(q, offsets):
    if offsets is not None and q.dim() != 3:
        raise ValueError(f"q must be [tokens, heads, dim] with offsets, got {q.dim()} dimensions")
    if offsets is None and q.dim() != 4:
        raise ValueError(f"q must be [batch, tokens, heads, dim] without offsets, got {q.dim()} dimensions")
    return 2 if offsets is None else 1


def _token_rows(t, name, dtype, device, shape, offsets):
    """The given buffer of token rows after its checks, or a new one.  Rows behind the last packed
    sequence keep what a given buffer holds; a new one's are zeros, so that what follows over all rows
    (a sum over tokens) meets no stale memory."""
    if t is None and offsets is not None:
        return torch.zeros(shape, dtype=dtype, device=device)
    return given_or_new(t, name, dtype, device, shape)


def _size(need: int) -> int:
    if need < 0:
        raise ValueError("a size is beyond what the library takes (dim_k <= 128, dim_v <= 256, 64 tokens' rows of "
                         "any argument less than 2^31 bytes from the first to the last, 2^23 groups of 64 tokens)")
    return need


def delta_rule_workspace(q, k, v, g, beta, offsets=None, backward: bool = False) -> int:
    """Bytes of workspace delta_rule_forward (or delta_rule_backward) takes for
    these tensors; it depends on their sizes alone."""
    lib = load_library()
    s = _shape(q, k, v, g, beta, 1.0, offsets, _lead(q, offsets))
    return _size((lib.delta_rule_backward_workspace if backward else lib.delta_rule_forward_workspace)(byref(s)))


def delta_rule_forward(q, k, v, g, beta, initial_state=None, scale: Optional[float] = None, offsets=None, o=None,
                       final_state=None, want_final: bool = True, workspace=None, stream=None) -> Tuple[object, object]:
    """(o, final_state) of the gated delta rule over sequences (see
    include/delta_rule.h): per value head, from S_0 = ``initial_state`` (zeros
    if None),

        S' = exp(g_t) S_{t-1},  u_t = beta_t (v_t - S'^T k_t),
        S_t = S' + k_t u_t^T,   o_t = scale S_t^T q_t

    ``q``, ``k`` [B, T, heads_k, dim_k] and ``v`` [B, T, heads_v, dim_v] are
    float32, bfloat16 or float16, of any token and head strides with a dense
    last axis and, where B > 1, the sequences one behind the other (slices of one
    projection are read where they lie); ``g`` (the
    decay's logarithm) and ``beta`` [B, T, heads_v] and the states
    [B, heads_v, dim_k, dim_v] are contiguous float32.  ``scale`` is
    dim_k ** -0.5 by default.  With ``offsets`` (int32 on the GPU, [S + 1]) the
    tokens are packed, [N, heads, dim] with sequence s in rows offsets[s] to
    offsets[s + 1] - 1; rows behind the last one's end keep what a given ``o``
    holds (with ``o`` given no fill is launched) and are zeros in a new one.
    ``final_state`` may be ``initial_state`` itself; ``want_final=False`` leaves
    it out (None).  The workspace is allocated here unless given."""
    lib = load_library()
    s = _shape(q, k, v, g, beta, scale, offsets, _lead(q, offsets))
    states = (s.n_seq, s.heads_v, s.dim_k, s.dim_v)
    dev = q.device
    with on_device(dev, stream):
        if initial_state is not None:
            check(initial_state, "initial_state", F32, dev, states)
        o = _token_rows(o, "o", q.dtype, dev, v.shape, offsets)
        if final_state is not None or want_final:
            final_state = given_or_new(final_state, "final_state", F32, dev, states)
        at, size, keep = space(_size(lib.delta_rule_forward_workspace(byref(s))), workspace, dev)
        _check("delta_rule_forward", lib.delta_rule_forward(
            byref(s), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), ptr(initial_state),
            o.data_ptr(), ptr(final_state), at, size, stream_ptr(dev, stream)))
    return o, final_state


def delta_rule_backward(q, k, v, g, beta, grad_o, initial_state=None, grad_final_state=None,
                        scale: Optional[float] = None, offsets=None, grad_q=None, grad_k=None, grad_v=None,
                        grad_g=None, grad_beta=None, grad_initial_state=None, workspace=None,
                        stream=None) -> Tuple[object, ...]:
    """(grad_q, grad_k, grad_v, grad_g, grad_beta, grad_initial_state): the
    gradients of sum(o * grad_o) + sum(final_state * grad_final_state) for
    delta_rule_forward's inputs, which are all it needs (the states are computed
    again).  ``grad_o`` has v's shape, its strides as free as q's;
    ``grad_final_state`` None means zeros.  Value heads that share a query and
    key head add up in grad_q and grad_k.  ``grad_initial_state`` is None where
    there is no initial state and no buffer is given for it."""
    lib = load_library()
    s = _shape(q, k, v, g, beta, scale, offsets, _lead(q, offsets), grad_o)
    states = (s.n_seq, s.heads_v, s.dim_k, s.dim_v)
    dev, dtype = q.device, q.dtype
    with on_device(dev, stream):
        if initial_state is not None:
            check(initial_state, "initial_state", F32, dev, states)
        if grad_final_state is not None:
            check(grad_final_state, "grad_final_state", F32, dev, states)
        grad_q = _token_rows(grad_q, "grad_q", dtype, dev, q.shape, offsets)
        grad_k = _token_rows(grad_k, "grad_k", dtype, dev, k.shape, offsets)
        grad_v = _token_rows(grad_v, "grad_v", dtype, dev, v.shape, offsets)
        grad_g = _token_rows(grad_g, "grad_g", F32, dev, g.shape, offsets)
        grad_beta = _token_rows(grad_beta, "grad_beta", F32, dev, g.shape, offsets)
        if grad_initial_state is not None or initial_state is not None:
            grad_initial_state = given_or_new(grad_initial_state, "grad_initial_state", F32, dev, states)
        at, size, keep = space(_size(lib.delta_rule_backward_workspace(byref(s))), workspace, dev)
        _check("delta_rule_backward", lib.delta_rule_backward(
            byref(s), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), ptr(initial_state),
            grad_o.data_ptr(), ptr(grad_final_state), grad_q.data_ptr(), grad_k.data_ptr(), grad_v.data_ptr(),
            grad_g.data_ptr(), grad_beta.data_ptr(), ptr(grad_initial_state), at, size, stream_ptr(dev, stream)))
    return grad_q, grad_k, grad_v, grad_g, grad_beta, grad_initial_state


def delta_rule_step(q, k, v, g, beta, states, slots=None, scale: Optional[float] = None, o=None, stream=None):
    """o [B, heads_v, dim_v] of one token for each row of a batch; the states
    [pool, heads_v, dim_k, dim_v] (contiguous float32) are updated where they
    are.  ``q``, ``k`` [B, heads_k, dim_k], ``v`` [B, heads_v, dim_v], ``g`` and
    ``beta`` [B, heads_v] are as in delta_rule_forward.  Row b's state is
    states[slots[b]] (int32 on the GPU), or states[b] without ``slots``.  A slot
    outside the pool (such as -1) makes the row idle: its o is zeros.  Rows that
    name one slot are taken one after the other, in the order of the rows."""
    lib = load_library()
    if q.dim() != 3:
        raise ValueError(f"q must be [batch, heads, dim], got {q.dim()} dimensions")
    s = _shape(q, k, v, g, beta, scale, None, 1)
    dev, rows = q.device, q.shape[0]
    if not isinstance(states, torch.Tensor) or states.dim() != 4:
        raise ValueError("states must be a tensor [pool, heads_v, dim_k, dim_v]")
    pool = states.shape[0]
    _ints(pool)
    check(states, "states", F32, dev, (pool, s.heads_v, s.dim_k, s.dim_v))
    if slots is not None:
        check(slots, "slots", torch.int32, dev, (rows,))
    elif pool < rows:
        raise ValueError(f"{rows} rows need as many states, got {pool}")
    with on_device(dev, stream):
        o = given_or_new(o, "o", q.dtype, dev, v.shape)
        _check("delta_rule_step", lib.delta_rule_step(
            byref(s), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), states.data_ptr(), pool,
            ptr(slots), o.data_ptr(), stream_ptr(dev, stream)))
    return o
