"""Tensor checks and pointer marshalling of the root-mean-square norm (include/rms_norm.h)."""
from __future__ import annotations

import math
from typing import Tuple

from ._lib import CFC_TYPE_F32, _check, _on_device, _stream_ptr, element_type, load_library


def _tensor(t, name, dtypes, device, shape):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes or not t.is_cuda or not t.is_contiguous() or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a contiguous tensor of {' or '.join(map(str, dtypes))} on "
                         f"{device or 'a GPU'} (got {t.dtype}, {t.device}, contiguous={t.is_contiguous()})")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _inputs(x, weight, residual):
    """(type, stream type, rows, width) after the checks that the forwards share."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a tensor [..., width]")
    kind = element_type(x, "x")
    _tensor(x, "x", (x.dtype,), None, None)
    width = x.shape[-1]
    _tensor(weight, "weight", (x.dtype,), x.device, (width,))
    stream_kind = kind
    if residual is not None:
        _tensor(residual, "residual", (x.dtype, torch.float32), x.device, x.shape)
        stream_kind = element_type(residual, "residual")
    return kind, stream_kind, math.prod(x.shape[:-1]), width


def _stream_out(h, x, residual):
    """The buffer of h = x + residual: a given one (residual itself among them), or a new one."""
    import torch
    if residual is None:
        if h is not None:
            raise ValueError("h needs a residual: without one it is x itself")
        return None
    if h is None:
        return torch.empty_like(residual)
    return _tensor(h, "h", (residual.dtype,), x.device, x.shape)


def rms_norm_forward(x, weight, eps: float, residual=None, y=None, h=None, rstd=None, want_rstd: bool = True,
                     stream=None) -> Tuple[object, object, object]:
    """(y, h, rstd) of rows x [..., width] (see include/rms_norm.h):
    h = x + residual rounded to the residual's type, rstd = 1 / sqrt(mean(h^2)
    + eps), y = h * rstd * weight in x's type.  x is float32, bfloat16 or
    float16, weight [width] of its type, residual of its type or float32; all
    contiguous.  ``h`` may be ``residual`` itself; without a residual h is x.
    rstd [...] is float32 (``want_rstd=False``: None)."""
    import torch
    lib = load_library()
    kind, stream_kind, rows, width = _inputs(x, weight, residual)
    with _on_device(x.device, stream):
        h = _stream_out(h, x, residual)
        y = torch.empty_like(x) if y is None else _tensor(y, "y", (x.dtype,), x.device, x.shape)
        if rstd is not None or want_rstd:
            rstd = (torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if rstd is None else
                    _tensor(rstd, "rstd", (torch.float32,), x.device, x.shape[:-1]))
        _check("rms_norm_forward", lib.rms_norm_forward(
            kind, stream_kind, rows, width, x.data_ptr(), _ptr(residual), weight.data_ptr(), float(eps), y.data_ptr(),
            _ptr(h), _ptr(rstd), _stream_ptr(x.device, stream)))
    return y, x if h is None else h, rstd


def rms_norm_forward_e4m3(x, weight, eps: float, residual=None, group: int = 0, y=None, scales=None, h=None,
                          rstd=None, stream=None) -> Tuple[object, object, object]:
    """(y, scales, h): rms_norm_forward's y in float8_e4m3fn with float32 scales
    [..., ceil(width / group)], y ~ value * scale: one for each ``group`` columns
    (a power of two from 16 to 512) or, with 0, for each row.  A scale is its
    columns' largest |y| / 448 (1 / 448 where all are zero).  ``rstd`` is written
    where a buffer is given for it."""
    import torch
    lib = load_library()
    kind, stream_kind, rows, width = _inputs(x, weight, residual)
    if group != 0 and (group < 16 or group > 512 or group & (group - 1)):
        raise ValueError(f"group must be 0 or a power of two from 16 to 512, got {group}")
    shape = (*x.shape[:-1], -(-width // group) if group else 1)
    with _on_device(x.device, stream):
        h = _stream_out(h, x, residual)
        e4m3 = torch.float8_e4m3fn
        y = (torch.empty(x.shape, dtype=e4m3, device=x.device) if y is None else
             _tensor(y, "y", (e4m3,), x.device, x.shape))
        scales = (torch.empty(shape, dtype=torch.float32, device=x.device) if scales is None else
                  _tensor(scales, "scales", (torch.float32,), x.device, shape))
        if rstd is not None:
            _tensor(rstd, "rstd", (torch.float32,), x.device, x.shape[:-1])
        _check("rms_norm_forward_e4m3", lib.rms_norm_forward_e4m3(
            kind, stream_kind, rows, width, x.data_ptr(), _ptr(residual), weight.data_ptr(), float(eps), int(group),
            y.data_ptr(), scales.data_ptr(), _ptr(h), _ptr(rstd), _stream_ptr(x.device, stream)))
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
    import torch
    lib = load_library()
    if not isinstance(grad_y, torch.Tensor) or grad_y.dim() < 1:
        raise ValueError("grad_y must be a tensor [..., width]")
    kind, dev, shape = element_type(grad_y, "grad_y"), grad_y.device, grad_y.shape
    _tensor(grad_y, "grad_y", (grad_y.dtype,), None, None)
    _tensor(h, "h", (grad_y.dtype, torch.float32), dev, shape)
    _tensor(weight, "weight", (grad_y.dtype,), dev, shape[-1:])
    _tensor(rstd, "rstd", (torch.float32,), dev, shape[:-1])
    if grad_h is not None:
        _tensor(grad_h, "grad_h", (h.dtype,), dev, shape)
    rows, width = math.prod(shape[:-1]), shape[-1]
    with _on_device(dev, stream):
        grad_x = torch.empty_like(h) if grad_x is None else _tensor(grad_x, "grad_x", (h.dtype,), dev, shape)
        grad_weight = (torch.empty((width,), dtype=torch.float32, device=dev) if grad_weight is None else
                       _tensor(grad_weight, "grad_weight", (torch.float32,), dev, (width,)))
        if workspace is None:
            workspace = torch.empty((rms_norm_backward_workspace(rows, width),), dtype=torch.uint8, device=dev)
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        _check("rms_norm_backward", lib.rms_norm_backward(
            kind, CFC_TYPE_F32 if h.dtype == torch.float32 else kind, rows, width, grad_y.data_ptr(), h.data_ptr(),
            weight.data_ptr(), rstd.data_ptr(), _ptr(grad_h), grad_x.data_ptr(), grad_weight.data_ptr(),
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_ptr(dev, stream)))
    return grad_x, grad_weight
