"""Tensor checks and pointer marshalling of the root-mean-square norm (include/rms_norm.h)."""
from __future__ import annotations

import math
from typing import Tuple

import torch

from ._lib import CFC_TYPE_F32, _check, load_library
from ._tensors import F32, check, element_type, given_or_new, on_device, ptr, space, stream_ptr

_E4M3 = torch.float8_e4m3fn


def _stream_type(t, name, like, kind, device, shape):
    """The type of a tensor of the residual stream: like's, or float32."""
    check(t, name, F32 if t.dtype == F32 else like.dtype, device, shape)
    return CFC_TYPE_F32 if t.dtype == F32 else kind


def _rows_of(x):
    """(device, shape) of x [..., width]."""
    element_type(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be a tensor [..., width]")
    check(x, "x", x.dtype, None)
    return x.device, x.shape


def _inputs(x, weight, residual, h):
    """(type, stream type, rows, width, buffer of h) after the checks that the forwards share."""
    kind, dev, shape = element_type(x, "x"), x.device, x.shape
    width = shape[-1]
    check(weight, "weight", x.dtype, dev, (width,))
    stream_kind = kind
    if residual is not None:
        stream_kind = _stream_type(residual, "residual", x, kind, dev, shape)
        if h is not residual:
            h = given_or_new(h, "h", residual.dtype, dev, shape, residual)
    elif h is not None:
        raise ValueError("h needs a residual: without one it is x itself")
    return kind, stream_kind, math.prod(shape[:-1]), width, h


def rms_norm_forward(x, weight, eps: float, residual=None, y=None, h=None, rstd=None, want_rstd: bool = True,
                     stream=None) -> Tuple[object, object, object]:
    """(y, h, rstd) of rows x [..., width] (see include/rms_norm.h):
    h = x + residual rounded to the residual's type, rstd = 1 / sqrt(mean(h^2)
    + eps), y = h * rstd * weight in x's type.  x is float32, bfloat16 or
    float16, weight [width] of its type, residual of its type or float32; all
    contiguous.  ``h`` may be ``residual`` itself; without a residual h is x.
    rstd [...] is float32 (``want_rstd=False``: None)."""
    lib = load_library()
    dev, shape = _rows_of(x)
    with on_device(dev, stream):
        kind, stream_kind, rows, width, h = _inputs(x, weight, residual, h)
        y = given_or_new(y, "y", x.dtype, dev, shape, x)
        if rstd is not None or want_rstd:
            rstd = given_or_new(rstd, "rstd", F32, dev, shape[:-1])
        _check("rms_norm_forward", lib.rms_norm_forward(
            kind, stream_kind, rows, width, x.data_ptr(), ptr(residual), weight.data_ptr(), eps, y.data_ptr(), ptr(h),
            ptr(rstd), stream_ptr(dev, stream)))
    return y, x if h is None else h, rstd


def rms_norm_forward_e4m3(x, weight, eps: float, residual=None, group: int = 0, y=None, scales=None, h=None,
                          rstd=None, stream=None) -> Tuple[object, object, object]:
    """(y, scales, h): rms_norm_forward's y in float8_e4m3fn with float32 scales
    [..., ceil(width / group)], y ~ value * scale: one for each ``group`` columns
    (a power of two from 16 to 512) or, with 0, for each row.  A scale is its
    columns' largest |y| / 448 (1 / 448 where all are zero).  ``rstd`` is written
    where a buffer is given for it."""
    lib = load_library()
    if group != 0 and (group < 16 or group > 512 or group & (group - 1)):
        raise ValueError(f"group must be 0 or a power of two from 16 to 512, got {group}")
    dev, shape = _rows_of(x)
    with on_device(dev, stream):
        kind, stream_kind, rows, width, h = _inputs(x, weight, residual, h)
        y = given_or_new(y, "y", _E4M3, dev, shape, x)
        scales = given_or_new(scales, "scales", F32, dev, shape[:-1] + (-(-width // group) if group else 1,))
        if rstd is not None:
            check(rstd, "rstd", F32, dev, shape[:-1])
        _check("rms_norm_forward_e4m3", lib.rms_norm_forward_e4m3(
            kind, stream_kind, rows, width, x.data_ptr(), ptr(residual), weight.data_ptr(), eps, group, y.data_ptr(),
            scales.data_ptr(), ptr(h), ptr(rstd), stream_ptr(dev, stream)))
    return y, scales, x if h is None else h


def rms_norm_backward_workspace(rows: int, width: int) -> int:
    """Bytes of workspace rms_norm_backward takes."""
    n = int(load_library().rms_norm_backward_workspace(rows, width))
    if n < 0:
        raise ValueError(f"invalid size rows={rows} width={width} (widths are 1 to 16384)")
    return n


def rms_norm_backward(grad_y, h, weight, rstd, grad_h=None, grad_x=None, grad_weight=None, workspace=None,
                      stream=None) -> Tuple[object, object]:
    """(grad_x, grad_weight) from rms_norm_forward's h and rstd: grad_x, of h's
    type, is the gradient of h and so of x and of the residual alike, with
    ``grad_h`` (what reaches h by itself, through the residual stream) added;
    it may be ``grad_h`` itself.  grad_weight [width] is float32.  The workspace
    is allocated here unless given."""
    lib = load_library()
    kind = element_type(grad_y, "grad_y")
    if grad_y.dim() < 1:
        raise ValueError("grad_y must be a tensor [..., width]")
    dev, shape = grad_y.device, grad_y.shape
    check(grad_y, "grad_y", grad_y.dtype, None)
    stream_kind = _stream_type(h, "h", grad_y, kind, dev, shape)
    rows, width = math.prod(shape[:-1]), shape[-1]
    check(weight, "weight", grad_y.dtype, dev, (width,))
    check(rstd, "rstd", F32, dev, shape[:-1])
    if grad_h is not None:
        check(grad_h, "grad_h", h.dtype, dev, shape)
    with on_device(dev, stream):
        grad_x = given_or_new(grad_x, "grad_x", h.dtype, dev, shape, h)
        grad_weight = given_or_new(grad_weight, "grad_weight", F32, dev, (width,))
        at, size, keep = space(rms_norm_backward_workspace(rows, width), workspace, dev)
        _check("rms_norm_backward", lib.rms_norm_backward(
            kind, stream_kind, rows, width, grad_y.data_ptr(), h.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
            ptr(grad_h), grad_x.data_ptr(), grad_weight.data_ptr(), at, size, stream_ptr(dev, stream)))
    return grad_x, grad_weight
