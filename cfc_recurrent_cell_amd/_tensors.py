"""What the bindings share: checks of tensors, streams, the current device.

A serving loop's calls are a few microseconds of GPU work, so the checks take
the short way where everything fits and say what does not only where it does
not.
"""
from __future__ import annotations

import contextlib

import torch

from ._lib import CFC_TYPE_BF16, CFC_TYPE_F16, CFC_TYPE_F32

TYPES = {torch.float32: CFC_TYPE_F32, torch.bfloat16: CFC_TYPE_BF16, torch.float16: CFC_TYPE_F16}
F32 = torch.float32
_HERE = contextlib.nullcontext()


def element_type(t, name: str) -> int:
    """The library's CFC_TYPE_* of a tensor's elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    kind = TYPES.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return kind


def check(t, name: str, dtype, device, shape=None):
    """t, if it is a contiguous tensor of that type on that GPU (of that shape)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {device or 'a GPU'} "
                         f"(got {t.dtype}, {t.device}, contiguous={t.is_contiguous()})")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def given_or_new(t, name: str, dtype, device, shape, like=None):
    """The buffer t after its checks, or a new one (as ``like``, a contiguous tensor of that
    shape, where there is one: 0.6 us less)."""
    if t is not None:
        return check(t, name, dtype, device, shape)
    if like is not None:
        return torch.empty_like(like, dtype=dtype)
    return torch.empty(shape, dtype=dtype, device=device)


def space(need: int, workspace, device):
    """(pointer, bytes, tensor) of the given workspace, or of a new one of `need` bytes."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def ptr(t):
    return None if t is None else t.data_ptr()


def stream_ptr(device, stream):
    # (the current stream's handle without making a torch.cuda.Stream: 0.1 against 2 us)
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def on_device(device, stream):
    """A context with ``device`` current, and ``stream`` too where one is given: what
    is allocated inside belongs to that stream, so memory freed while its kernels
    still run is not handed to another one."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)  # makes the stream's device current
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)
