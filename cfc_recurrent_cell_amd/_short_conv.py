"""Tensor checks and pointer marshalling of the short causal convolution (include/short_conv.h)."""
from __future__ import annotations

from ctypes import byref
from typing import Optional, Tuple

import torch

from ._lib import ShortConvShape, _check, load_library
from ._sequences import _ints, given_or_cleared, lead_of, row_stride, sequences_of, slots_of
from ._tensors import F32, check, element_type, given_or_new, on_device, ptr, space, stream_ptr


def _shape(x, weight, bias, activation, lead, offsets, grad_y=None):
    kind, dtype, dev = element_type(x, "x"), x.dtype, x.device
    channels = x.shape[-1]
    stride = row_stride(x, "x", lead, dtype, dev, x.shape)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a tensor [channels, width]")
    width = weight.shape[1]
    check(weight, "weight", dtype, dev, (channels, width))
    if bias is not None:
        check(bias, "bias", dtype, dev, (channels,))
    if activation not in ("silu", None):
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    if not 2 <= width <= 4:
        raise ValueError(f"weight has {width} taps, expected 2, 3 or 4")
    if channels < 1:
        raise ValueError("x must have at least one channel")
    grad_stride = 0 if grad_y is None else row_stride(grad_y, "grad_y", lead, dtype, dev, x.shape)
    count, length, tokens, at = sequences_of(x, lead, offsets)
    _ints(channels)
    return ShortConvShape(kind, count, length, tokens, at, channels, width, int(activation is not None), 0,
                          stride, grad_stride)


def _size(need: int) -> int:
    if need < 0:
        raise ValueError("a size is beyond what the library takes (at most 2^31 - 2^16 tokens)")
    return need


def short_conv_forward(x, weight, bias=None, initial_state=None, activation: Optional[str] = "silu", offsets=None,
                       y=None, final_state=None, want_final: bool = True, stream=None) -> Tuple[object, object]:
    """(y, final_state) of the causal convolution of each channel over sequences (see
    include/short_conv.h):

        p_t = bias + sum_j weight[:, j] x_{t - width + 1 + j},   y_t = p_t sigmoid(p_t)

    (``activation=None``: y = p).  ``x`` [B, T, channels] is float32, bfloat16 or float16, of
    any token stride with a dense last axis and, where B > 1, the sequences one behind the
    other (a slice of a projection is read where it lies); ``weight`` [channels, width] with a
    width of 2 to 4, ``bias`` [channels] and the states [B, width - 1, channels] (the inputs
    before the first token, the oldest first; None: zeros) are contiguous and of x's type.
    With ``offsets`` (int32 on the GPU, [S + 1]) the tokens are packed, [N, channels] with
    sequence s in rows offsets[s] to offsets[s + 1] - 1; rows behind the last one's end keep
    what a given ``y`` holds and are zeros in a new one.  ``final_state`` may be
    ``initial_state`` itself; ``want_final=False`` leaves it out (None)."""
    lib = load_library()
    s = _shape(x, weight, bias, activation, lead_of(x, offsets), offsets)
    states, dev, dtype = (s.n_seq, s.width - 1, s.channels), x.device, x.dtype
    with on_device(dev, stream):
        if initial_state is not None:
            check(initial_state, "initial_state", dtype, dev, states)
        y = given_or_cleared(s, 1, y, "y", dtype, dev, x.shape)
        if final_state is not None or want_final:
            final_state = given_or_new(final_state, "final_state", dtype, dev, states)
        _check("short_conv_forward", lib.short_conv_forward(
            byref(s), x.data_ptr(), weight.data_ptr(), ptr(bias), ptr(initial_state), y.data_ptr(), ptr(final_state),
            stream_ptr(dev, stream)))
    return y, final_state


def short_conv_backward_workspace(x, weight, offsets=None) -> int:
    """Bytes of workspace short_conv_backward takes for these tensors; it depends on their
    sizes alone."""
    s = _shape(x, weight, None, None, lead_of(x, offsets), offsets)
    return _size(int(load_library().short_conv_backward_workspace(byref(s))))


def short_conv_backward(x, weight, grad_y, bias=None, initial_state=None, grad_final_state=None,
                        activation: Optional[str] = "silu", offsets=None, grad_x=None, grad_weight=None,
                        grad_bias=None, grad_initial_state=None, workspace=None, stream=None) -> Tuple[object, ...]:
    """(grad_x, grad_weight, grad_bias, grad_initial_state): the gradients of
    sum(y * grad_y) + sum(final_state * grad_final_state) for short_conv_forward's inputs,
    which are all it needs.  ``grad_y`` has x's shape, its stride as free as x's;
    ``grad_final_state`` None means zeros.  grad_weight and grad_bias are float32; grad_bias is
    None where there is no bias, grad_initial_state where there is no initial state, and no
    buffer is given for it.  The workspace is allocated here unless given."""
    lib = load_library()
    s = _shape(x, weight, bias, activation, lead_of(x, offsets), offsets, grad_y)
    states, dev, dtype = (s.n_seq, s.width - 1, s.channels), x.device, x.dtype
    with on_device(dev, stream):
        for t, name in ((initial_state, "initial_state"), (grad_final_state, "grad_final_state")):
            if t is not None:
                check(t, name, dtype, dev, states)
        grad_x = given_or_cleared(s, 1, grad_x, "grad_x", dtype, dev, x.shape)
        grad_weight = given_or_new(grad_weight, "grad_weight", F32, dev, (s.channels, s.width))
        if grad_bias is not None or bias is not None:
            grad_bias = given_or_new(grad_bias, "grad_bias", F32, dev, (s.channels,))
        if grad_initial_state is not None or initial_state is not None:
            grad_initial_state = given_or_new(grad_initial_state, "grad_initial_state", dtype, dev, states)
        at, size, keep = space(_size(lib.short_conv_backward_workspace(byref(s))), workspace, dev)
        _check("short_conv_backward", lib.short_conv_backward(
            byref(s), x.data_ptr(), weight.data_ptr(), ptr(bias), ptr(initial_state), grad_y.data_ptr(),
            ptr(grad_final_state), grad_x.data_ptr(), grad_weight.data_ptr(), ptr(grad_bias), ptr(grad_initial_state),
            at, size, stream_ptr(dev, stream)))
    return grad_x, grad_weight, grad_bias, grad_initial_state


def short_conv_step(x, weight, states, slots=None, bias=None, activation: Optional[str] = "silu", y=None, stream=None):
    """y [B, channels] of one token for each row of a batch; the states
    [pool, width - 1, channels] (contiguous, of x's type) are updated where they are.
    ``x`` [B, channels], ``weight`` and ``bias`` are as in short_conv_forward.  Row b's state
    is states[slots[b]] (int32 on the GPU), or states[b] without ``slots``.  A slot outside
    the pool (such as -1) makes the row idle: its y is zeros.  Rows that name one slot are
    taken one after the other, in the order of the rows."""
    lib = load_library()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a tensor [batch, channels]")
    s = _shape(x, weight, bias, activation, 1, None)
    dev, rows = x.device, x.shape[0]
    pool = slots_of(slots, rows, states, (s.width - 1, s.channels), x.dtype, dev)
    with on_device(dev, stream):
        y = given_or_new(y, "y", x.dtype, dev, x.shape, x if x.is_contiguous() else None)
        _check("short_conv_step", lib.short_conv_step(
            byref(s), x.data_ptr(), weight.data_ptr(), ptr(bias), states.data_ptr(), pool, ptr(slots), y.data_ptr(),
            stream_ptr(dev, stream)))
    return y
