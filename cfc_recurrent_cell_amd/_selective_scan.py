"""Tensor checks and pointer marshalling of the selective scan (include/selective_scan.h)."""
from __future__ import annotations

from ctypes import byref
from typing import Tuple

import torch

from ._delta_rule import _rows
from ._lib import SelectiveScanShape, _check, load_library
from ._sequences import _ints, given_or_cleared, lead_of, row_stride, sequences_of, slots_of
from ._tensors import F32, check, element_type, given_or_new, on_device, ptr, space, stream_ptr

# SELECTIVE_SCAN_CLEAR_* of include/selective_scan.h
_CLEAR_Y, _CLEAR_X, _CLEAR_DT, _CLEAR_B, _CLEAR_C, _CLEAR_Z = 1, 1, 2, 4, 8, 16


def _shape(x, dt, a, b, c, d, z, dt_bias, softplus, lead, offsets, grad_y=None):
    kind, dtype, dev, n = element_type(x, "x"), x.dtype, x.device, x.shape
    channels = n[-1]
    strides = [row_stride(x, "x", lead, dtype, dev, n), row_stride(dt, "dt", lead, dtype, dev, n)]
    strides += [0 if t is None else row_stride(t, name, lead, dtype, dev, n)
                for t, name in ((z, "z"), (grad_y, "grad_y"))]
    bs = _rows(b, "b", lead, dtype, dev)
    cs = _rows(c, "c", lead, dtype, dev, b.shape)
    if b.shape[:lead] != n[:lead]:
        raise ValueError(f"b has shape {tuple(b.shape)}, expected {tuple(n[:lead])} tokens as x has")
    groups, state = b.shape[-2], b.shape[-1]
    if groups < 1 or channels < 1 or channels % groups:
        raise ValueError(f"x's {channels} channels are no multiple of b's {groups} groups")
    if not 1 <= state <= 64:
        raise ValueError(f"b has states of {state} elements, expected 1 to 64")
    check(a, "a", F32, dev, (channels, state))
    for t, name in ((d, "d"), (dt_bias, "dt_bias")):
        if t is not None:
            check(t, name, F32, dev, (channels,))
    count, length, tokens, at = sequences_of(x, lead, offsets)
    _ints(channels)
    return SelectiveScanShape(kind, count, length, tokens, at, channels, groups, state, int(bool(softplus)), 0, *strides,
                              *bs, *cs)


def _size(need: int) -> int:
    if need < 0:
        raise ValueError("a size is beyond what the library takes (at most 2^31 - 2^16 tokens, and 2^31 elements of b)")
    return need


def selective_scan_forward(x, dt, a, b, c, d=None, z=None, dt_bias=None, initial_state=None, softplus: bool = True,
                           offsets=None, y=None, final_state=None, want_final: bool = True,
                           stream=None) -> Tuple[object, object]:
    """(y, final_state) of the selective scan over sequences (see
    include/selective_scan.h): per channel, from h_0 = ``initial_state`` (zeros if None),

        D_t = softplus(dt_t + dt_bias),  h_t = exp(D_t a) h_{t-1} + D_t x_t b_t,
        y_t = (sum_n c_t h_t + d x_t) z_t sigmoid(z_t)

    (``softplus=False``: D = dt + dt_bias; without ``z`` no gate, without ``d`` no skip).
    ``x``, ``dt``, ``z`` [B, T, channels] and ``b``, ``c`` [B, T, groups, state] are float32,
    bfloat16 or float16, of any token and group strides with a dense last axis and, where
    B > 1, the sequences one behind the other (slices of projections are read where they
    lie); ``a`` [channels, state], ``d`` and ``dt_bias`` [channels] and the states
    [B, channels, state] are contiguous float32.  A group of channels / groups
    neighbouring channels shares b and c.  With ``offsets`` (int32 on the GPU, [S + 1]) the
    tokens are packed, [N, ...] with sequence s in rows offsets[s] to offsets[s + 1] - 1;
    rows behind the last one's end keep what a given ``y`` holds and are zeros in a new one.
    ``final_state`` may be ``initial_state`` itself; ``want_final=False`` leaves it out
    (None)."""
    lib = load_library()
    s = _shape(x, dt, a, b, c, d, z, dt_bias, softplus, lead_of(x, offsets), offsets)
    states, dev = (s.n_seq, s.channels, s.state), x.device
    with on_device(dev, stream):
        if initial_state is not None:
            check(initial_state, "initial_state", F32, dev, states)
        y = given_or_cleared(s, _CLEAR_Y, y, "y", x.dtype, dev, x.shape)
        if final_state is not None or want_final:
            final_state = given_or_new(final_state, "final_state", F32, dev, states)
        _check("selective_scan_forward", lib.selective_scan_forward(
            byref(s), x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), ptr(d), ptr(z),
            ptr(dt_bias), ptr(initial_state), y.data_ptr(), ptr(final_state), stream_ptr(dev, stream)))
    return y, final_state


def selective_scan_backward_workspace(x, dt, a, b, c, offsets=None) -> int:
    """Bytes of workspace selective_scan_backward takes for these tensors; it depends on
    their sizes alone."""
    s = _shape(x, dt, a, b, c, None, None, None, True, lead_of(x, offsets), offsets)
    return _size(int(load_library().selective_scan_backward_workspace(byref(s))))


def selective_scan_backward(x, dt, a, b, c, grad_y, d=None, z=None, dt_bias=None, initial_state=None,
                            grad_final_state=None, softplus: bool = True, offsets=None, grad_x=None, grad_dt=None,
                            grad_a=None, grad_b=None, grad_c=None, grad_d=None, grad_z=None, grad_dt_bias=None,
                            grad_initial_state=None, workspace=None, stream=None) -> Tuple[object, ...]:
    """(grad_x, grad_dt, grad_a, grad_b, grad_c, grad_d, grad_z, grad_dt_bias,
    grad_initial_state): the gradients of sum(y * grad_y) + sum(final_state *
    grad_final_state) for selective_scan_forward's inputs, which are all it needs (the
    states are computed again).  ``grad_y`` has x's shape, its stride as free as x's;
    ``grad_final_state`` None means zeros.  grad_a, grad_d and grad_dt_bias are float32,
    the others of their input's type; channels of a group add up in grad_b and grad_c.
    Those of inputs that are not given (d, z, dt_bias, initial_state) are None, where no
    buffer is given for them.  The workspace is allocated here unless given."""
    lib = load_library()
    s = _shape(x, dt, a, b, c, d, z, dt_bias, softplus, lead_of(x, offsets), offsets, grad_y)
    states, dev, dtype = (s.n_seq, s.channels, s.state), x.device, x.dtype
    if z is None and grad_z is not None:
        raise ValueError("grad_z needs z")
    with on_device(dev, stream):
        for t, name in ((initial_state, "initial_state"), (grad_final_state, "grad_final_state")):
            if t is not None:
                check(t, name, F32, dev, states)
        grad_x = given_or_cleared(s, _CLEAR_X, grad_x, "grad_x", dtype, dev, x.shape)
        grad_dt = given_or_cleared(s, _CLEAR_DT, grad_dt, "grad_dt", dtype, dev, x.shape)
        grad_a = given_or_new(grad_a, "grad_a", F32, dev, a.shape)
        grad_b = given_or_cleared(s, _CLEAR_B, grad_b, "grad_b", dtype, dev, b.shape)
        grad_c = given_or_cleared(s, _CLEAR_C, grad_c, "grad_c", dtype, dev, b.shape)
        if grad_d is not None or d is not None:
            grad_d = given_or_new(grad_d, "grad_d", F32, dev, (s.channels,))
        if z is not None:
            grad_z = given_or_cleared(s, _CLEAR_Z, grad_z, "grad_z", dtype, dev, x.shape)
        if grad_dt_bias is not None or dt_bias is not None:
            grad_dt_bias = given_or_new(grad_dt_bias, "grad_dt_bias", F32, dev, (s.channels,))
        if grad_initial_state is not None or initial_state is not None:
            grad_initial_state = given_or_new(grad_initial_state, "grad_initial_state", F32, dev, states)
        at, size, keep = space(_size(lib.selective_scan_backward_workspace(byref(s))), workspace, dev)
        _check("selective_scan_backward", lib.selective_scan_backward(
            byref(s), x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), ptr(d), ptr(z),
            ptr(dt_bias), ptr(initial_state), grad_y.data_ptr(), ptr(grad_final_state), grad_x.data_ptr(),
            grad_dt.data_ptr(), grad_a.data_ptr(), grad_b.data_ptr(), grad_c.data_ptr(), ptr(grad_d), ptr(grad_z),
            ptr(grad_dt_bias), ptr(grad_initial_state), at, size, stream_ptr(dev, stream)))
    return grad_x, grad_dt, grad_a, grad_b, grad_c, grad_d, grad_z, grad_dt_bias, grad_initial_state


def selective_scan_step(x, dt, a, b, c, states, slots=None, d=None, z=None, dt_bias=None, softplus: bool = True, y=None,
                        stream=None):
    """y [B, channels] of one token for each row of a batch; the states
    [pool, channels, state] (contiguous float32) are updated where they are.  ``x``, ``dt``,
    ``z`` [B, channels], ``b``, ``c`` [B, groups, state] and the others are as in
    selective_scan_forward.  Row r's state is states[slots[r]] (int32 on the GPU), or
    states[r] without ``slots``.  A slot outside the pool (such as -1) makes the row idle: its
    y is zeros.  Rows that name one slot are taken one after the other, in the order of the
    rows."""
    lib = load_library()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a tensor [batch, channels]")
    s = _shape(x, dt, a, b, c, d, z, dt_bias, softplus, 1, None)
    dev, rows = x.device, x.shape[0]
    pool = slots_of(slots, rows, states, (s.channels, s.state), F32, dev)
    with on_device(dev, stream):
        y = given_or_new(y, "y", x.dtype, dev, x.shape, x if x.is_contiguous() else None)
        _check("selective_scan_step", lib.selective_scan_step(
            byref(s), x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), ptr(d), ptr(z),
            ptr(dt_bias), states.data_ptr(), pool, ptr(slots), y.data_ptr(), stream_ptr(dev, stream)))
    return y
