"""Tensor checks and pointer marshalling of the layer norm (include/layer_norm.h)."""
from __future__ import annotations

import math
from typing import Tuple

from ._lib import _check, load_library
from ._rms_norm import _inputs, _rows_of, _stream_type
from ._tensors import F32, check, element_type, given_or_new, on_device, ptr, space, stream_ptr


def layer_norm_forward(x, weight, bias, eps: float, residual=None, y=None, h=None, mean=None, rstd=None,
                       want_stats: bool = True, stream=None) -> Tuple[object, object, object, object]:
    """(y, h, mean, rstd) of rows x [..., width] (see include/layer_norm.h):
    h = x + residual rounded to the residual's type, a row's mean and
    rstd = 1 / sqrt(mean((h - mean)^2) + eps), y = (h - mean) * rstd * weight + bias
    in x's type.  x is float32, bfloat16 or float16, weight and bias [width] of its
    type (bias None: zeros), residual of its type or float32; all contiguous.  ``h``
    may be ``residual`` itself; without a residual h is x.  mean and rstd [...] are
    float32 (``want_stats=False``: None where no buffer is given)."""
    lib = load_library()
    dev, shape = _rows_of(x)
    with on_device(dev, stream):
        kind, stream_kind, rows, width, h = _inputs(x, weight, residual, h)
        if bias is not None:
            check(bias, "bias", x.dtype, dev, (width,))
        y = given_or_new(y, "y", x.dtype, dev, shape, x)
        if mean is not None or want_stats:
            mean = given_or_new(mean, "mean", F32, dev, shape[:-1])
        if rstd is not None or want_stats:
            rstd = given_or_new(rstd, "rstd", F32, dev, shape[:-1])
        _check("layer_norm_forward", lib.layer_norm_forward(
            kind, stream_kind, rows, width, x.data_ptr(), ptr(residual), weight.data_ptr(), ptr(bias), eps,
            y.data_ptr(), ptr(h), ptr(mean), ptr(rstd), stream_ptr(dev, stream)))
    return y, x if h is None else h, mean, rstd


def layer_norm_backward_workspace(rows: int, width: int) -> int:
    """Bytes of workspace layer_norm_backward takes."""
    n = int(load_library().layer_norm_backward_workspace(rows, width))
    if n < 0:
        raise ValueError(f"invalid size rows={rows} width={width} (widths are 1 to 16384)")
    return n


def layer_norm_backward(grad_y, h, weight, mean, rstd, grad_h=None, grad_x=None, grad_weight=None, grad_bias=None,
                        want_bias: bool = True, workspace=None, stream=None) -> Tuple[object, object, object]:
    """(grad_x, grad_weight, grad_bias) from layer_norm_forward's h, mean and rstd:
    grad_x, of h's type, is the gradient of h and so of x and of the residual alike,
    with ``grad_h`` (what reaches h by itself, through the residual stream) added; it
    may be ``grad_h`` itself.  grad_weight and grad_bias [width] are float32
    (``want_bias=False``: None where no buffer is given).  The workspace is allocated
    here unless given."""
    lib = load_library()
    kind = element_type(grad_y, "grad_y")
    if grad_y.dim() < 1:
        raise ValueError("grad_y must be a tensor [..., width]")
    dev, shape = grad_y.device, grad_y.shape
    check(grad_y, "grad_y", grad_y.dtype, None)
    stream_kind = _stream_type(h, "h", grad_y, kind, dev, shape)
    rows, width = math.prod(shape[:-1]), shape[-1]
    check(weight, "weight", grad_y.dtype, dev, (width,))
    check(mean, "mean", F32, dev, shape[:-1])
    check(rstd, "rstd", F32, dev, shape[:-1])
    if grad_h is not None:
        check(grad_h, "grad_h", h.dtype, dev, shape)
    with on_device(dev, stream):
        grad_x = given_or_new(grad_x, "grad_x", h.dtype, dev, shape, h)
        grad_weight = given_or_new(grad_weight, "grad_weight", F32, dev, (width,))
        if grad_bias is not None or want_bias:
            grad_bias = given_or_new(grad_bias, "grad_bias", F32, dev, (width,))
        at, size, keep = space(layer_norm_backward_workspace(rows, width), workspace, dev)
        _check("layer_norm_backward", lib.layer_norm_backward(
            kind, stream_kind, rows, width, grad_y.data_ptr(), h.data_ptr(), weight.data_ptr(), mean.data_ptr(),
            rstd.data_ptr(), ptr(grad_h), grad_x.data_ptr(), grad_weight.data_ptr(), ptr(grad_bias), at, size,
            stream_ptr(dev, stream)))
    return grad_x, grad_weight, grad_bias
