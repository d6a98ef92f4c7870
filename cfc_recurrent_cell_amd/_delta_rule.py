"""Tensor checks and pointer marshalling of the gated delta rule (include/delta_rule.h)."""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

from ._lib import DeltaRuleShape, _check, _on_device, _stream_ptr, element_type, load_library


def _tensor(t, name, dtype, device, shape):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous() or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {device or 'a GPU'} "
                         f"(got {t.dtype}, {t.device}, contiguous={t.is_contiguous()})")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _rows(t, name, lead, like=None, shape=None):
    """(token stride, head stride) of t [*lead, heads, dim], rows numbered along its leading axes."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dim() != lead + 2 or (like is not None and (t.dtype != like.dtype or t.device != like.device)):
        raise ValueError(f"{name} must be a {lead + 2}-dimensional tensor on a GPU, of q's type and device "
                         f"(got {t.dim()} dimensions, {t.dtype}, {t.device})")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    n = t.shape
    if t.numel() == 0:
        return 0, 0
    if n[-1] > 1 and st[-1] != 1:
        raise ValueError(f"{name}'s last axis must be dense (its stride is {st[-1]})")
    if lead == 1:
        return st[0], st[1]
    if n[1] == 1:
        return st[0], st[2]
    if n[0] > 1 and n[1] > 1 and st[0] != n[1] * st[1]:
        raise ValueError(f"{name}'s sequences must lie one behind the other (strides {st}): make it contiguous")
    return st[1], st[2]


def _shape(q, k, v, g, beta, scale, offsets, lead, grad_o=None):
    import torch
    s = DeltaRuleShape()
    s.q_stride_t, s.q_stride_h = _rows(q, "q", lead)
    s.type = element_type(q, "q")
    s.k_stride_t, s.k_stride_h = _rows(k, "k", lead, q, q.shape)
    s.v_stride_t, s.v_stride_h = _rows(v, "v", lead, q)
    n = q.shape
    if v.shape[:lead] != n[:lead]:
        raise ValueError(f"v has shape {tuple(v.shape)}, expected {tuple(n[:lead])} tokens as q has")
    if grad_o is not None:
        s.go_stride_t, s.go_stride_h = _rows(grad_o, "grad_o", lead, q, v.shape)
    s.heads_k, s.dim_k = n[lead:]
    s.heads_v, s.dim_v = v.shape[lead:]
    if s.heads_k < 1 or s.heads_v % s.heads_k:
        raise ValueError(f"v's {s.heads_v} heads are no multiple of q's {s.heads_k}")
    gates = v.shape[:lead + 1]
    _tensor(g, "g", torch.float32, q.device, gates)
    _tensor(beta, "beta", torch.float32, q.device, gates)
    s.scale = s.dim_k ** -0.5 if scale is None else float(scale)
    s.n_tokens = n[0] if lead == 1 else n[0] * n[1]
    if offsets is not None:
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError("offsets must be a vector of the sequences' beginnings and the last one's end")
        _tensor(offsets, "offsets", torch.int32, q.device, offsets.shape)
        s.n_seq = offsets.numel() - 1
        s.offsets = offsets.data_ptr()
    elif lead == 2:
        s.n_seq, s.seq_len = n[0], n[1]
    return s


def _lead(q, offsets):
    if offsets is not None and q.dim() != 3:
        raise ValueError(f"q must be [tokens, heads, dim] with offsets, got {q.dim()} dimensions")
    if offsets is None and q.dim() != 4:
        raise ValueError(f"q must be [batch, tokens, heads, dim] without offsets, got {q.dim()} dimensions")
    return 2 if offsets is None else 1


def _space(need, workspace, device, what):
    import torch
    if need < 0:
        raise ValueError(f"{what}: a size is beyond what the library takes (dim_k <= 128, dim_v <= 256)")
    if workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _ptr(t):
    return t.data_ptr() if t is not None else None


def delta_rule_workspace(q, k, v, g, beta, offsets=None, backward: bool = False) -> int:
    """Bytes of workspace delta_rule_forward (or delta_rule_backward) takes for
    these tensors; it depends on their sizes alone."""
    lib = load_library()
    s = _shape(q, k, v, g, beta, 1.0, offsets, _lead(q, offsets))
    n = int((lib.delta_rule_backward_workspace if backward else lib.delta_rule_forward_workspace)(ctypes.byref(s)))
    if n < 0:
        raise ValueError("a size is beyond what the library takes (dim_k <= 128, dim_v <= 256)")
    return n


def delta_rule_forward(q, k, v, g, beta, initial_state=None, scale: Optional[float] = None, offsets=None, o=None,
                       final_state=None, want_final: bool = True, workspace=None, stream=None) -> Tuple[object, object]:
    """(o, final_state) of the gated delta rule over sequences (see
    include/delta_rule.h): per value head, from S_0 = ``initial_state`` (zeros
    if None),

        S' = exp(g_t) S_{t-1},  u_t = beta_t (v_t - S'^T k_t),
        S_t = S' + k_t u_t^T,   o_t = scale S_t^T q_t

    ``q``, ``k`` [B, T, heads_k, dim_k] and ``v`` [B, T, heads_v, dim_v] are
    float32, bfloat16 or float16, of any token and head strides with a dense
    last axis (slices of one projection are read where they lie); ``g`` (the
    decay's logarithm) and ``beta`` [B, T, heads_v] and the states
    [B, heads_v, dim_k, dim_v] are contiguous float32.  ``scale`` is
    dim_k ** -0.5 by default.  With ``offsets`` (int32 on the GPU, [S + 1]) the
    tokens are packed, [N, heads, dim] with sequence s in rows offsets[s] to
    offsets[s + 1] - 1; rows behind the last one's end keep what ``o`` held.
    ``final_state`` may be ``initial_state`` itself; ``want_final=False`` leaves
    it out (None).  The workspace is allocated here unless given."""
    import torch
    lib = load_library()
    lead = _lead(q, offsets)
    s = _shape(q, k, v, g, beta, scale, offsets, lead)
    states = (s.n_seq, s.heads_v, s.dim_k, s.dim_v)
    dev = q.device
    with _on_device(dev, stream):
        if initial_state is not None:
            _tensor(initial_state, "initial_state", torch.float32, dev, states)
        if o is None:
            o = torch.empty(v.shape, dtype=q.dtype, device=dev)
        _tensor(o, "o", q.dtype, dev, v.shape)
        if final_state is None and want_final:
            final_state = torch.empty(states, dtype=torch.float32, device=dev)
        if final_state is not None:
            _tensor(final_state, "final_state", torch.float32, dev, states)
        ws, ws_bytes, keep = _space(int(lib.delta_rule_forward_workspace(ctypes.byref(s))), workspace, dev,
                                    "delta_rule_forward")
        _check("delta_rule_forward", lib.delta_rule_forward(
            ctypes.byref(s), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            _ptr(initial_state), o.data_ptr(), _ptr(final_state), ws, ws_bytes, _stream_ptr(dev, stream)))
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
    import torch
    lib = load_library()
    lead = _lead(q, offsets)
    s = _shape(q, k, v, g, beta, scale, offsets, lead, grad_o)
    states = (s.n_seq, s.heads_v, s.dim_k, s.dim_v)
    dev = q.device
    with _on_device(dev, stream):
        for t, name in ((initial_state, "initial_state"), (grad_final_state, "grad_final_state")):
            if t is not None:
                _tensor(t, name, torch.float32, dev, states)

        def out(t, name, shape, dtype):
            # rows behind the last sequence have no gradient, and keep what a given buffer holds
            if t is None:
                make = torch.empty if offsets is None or name == "grad_initial_state" else torch.zeros
                return make(shape, dtype=dtype, device=dev)
            return _tensor(t, name, dtype, dev, shape)

        grad_q = out(grad_q, "grad_q", q.shape, q.dtype)
        grad_k = out(grad_k, "grad_k", k.shape, q.dtype)
        grad_v = out(grad_v, "grad_v", v.shape, q.dtype)
        grad_g = out(grad_g, "grad_g", g.shape, torch.float32)
        grad_beta = out(grad_beta, "grad_beta", g.shape, torch.float32)
        if grad_initial_state is not None or initial_state is not None:
            grad_initial_state = out(grad_initial_state, "grad_initial_state", states, torch.float32)
        ws, ws_bytes, keep = _space(int(lib.delta_rule_backward_workspace(ctypes.byref(s))), workspace, dev,
                                    "delta_rule_backward")
        _check("delta_rule_backward", lib.delta_rule_backward(
            ctypes.byref(s), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            _ptr(initial_state), grad_o.data_ptr(), _ptr(grad_final_state), grad_q.data_ptr(), grad_k.data_ptr(),
            grad_v.data_ptr(), grad_g.data_ptr(), grad_beta.data_ptr(), _ptr(grad_initial_state), ws, ws_bytes,
            _stream_ptr(dev, stream)))
    return grad_q, grad_k, grad_v, grad_g, grad_beta, grad_initial_state


def delta_rule_step(q, k, v, g, beta, states, slots=None, scale: Optional[float] = None, o=None, stream=None):
    """o [B, heads_v, dim_v] of one token for each row of a batch; the states
    [pool, heads_v, dim_k, dim_v] (contiguous float32) are updated where they
    are.  ``q``, ``k`` [B, heads_k, dim_k], ``v`` [B, heads_v, dim_v], ``g`` and
    ``beta`` [B, heads_v] are as in delta_rule_forward.  Row b's state is
    states[slots[b]] (int32 on the GPU), or states[b] without ``slots``.  A slot
    outside the pool (such as -1) makes the row idle: its o is zeros.  Rows that
    name one slot are taken one after the other, in the order of the rows."""
    import torch
    lib = load_library()
    if q.dim() != 3:
        raise ValueError(f"q must be [batch, heads, dim], got {q.dim()} dimensions")
    s = _shape(q, k, v, g, beta, scale, None, 1)
    dev = q.device
    if not isinstance(states, torch.Tensor) or states.dim() != 4:
        raise ValueError("states must be a tensor [pool, heads_v, dim_k, dim_v]")
    pool = states.shape[0]
    _tensor(states, "states", torch.float32, dev, (pool, s.heads_v, s.dim_k, s.dim_v))
    if slots is not None:
        _tensor(slots, "slots", torch.int32, dev, (s.n_tokens,))
    elif pool < s.n_tokens:
        raise ValueError(f"{s.n_tokens} rows need as many states, got {pool}")
    with _on_device(dev, stream):
        if o is None:
            o = torch.empty(v.shape, dtype=q.dtype, device=dev)
        _tensor(o, "o", q.dtype, dev, v.shape)
        _check("delta_rule_step", lib.delta_rule_step(
            ctypes.byref(s), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            states.data_ptr(), pool, _ptr(slots), o.data_ptr(), _stream_ptr(dev, stream)))
    return o
