"""Tensor checks and pointer marshalling of the gradients' norm and clipping (include/grad_norm.h)."""
from __future__ import annotations

from ctypes import c_uint64

import torch

from ._lib import GradTensor, _check, load_library
from ._tensors import F32, TYPES, check, element_type, given_or_new, on_device, space, stream_ptr


def _tensors(grads, out, norm):
    """(array of the library's descriptions, device) of the gradients and their outputs."""
    if isinstance(grads, torch.Tensor):
        raise TypeError("grads must be a list of tensors, not a tensor")
    grads = list(grads)
    if out is None:
        outs = grads
    else:
        outs = list(out)
        if len(outs) != len(grads):
            raise ValueError(f"out has {len(outs)} tensors, grads {len(grads)}")
    if not grads and norm is None:
        raise ValueError("grads must have at least one tensor, where no buffer is given for the norm")
    if not grads:
        check(norm, "norm", F32, None, ())
    first = grads[0] if grads else norm
    if not isinstance(first, torch.Tensor):
        raise TypeError("grads[0] must be a torch.Tensor")
    dev = first.device
    flat = []  # the descriptions' words: a tensor's are set at once, and not field by field
    for i, (g, o) in enumerate(zip(grads, outs)):
        # (the short way: what does not fit is named below)
        if not (isinstance(g, torch.Tensor) and g.is_cuda and g.device == dev and g.is_contiguous() and g.dtype in TYPES):
            element_type(g, f"grads[{i}]")
            check(g, f"grads[{i}]", g.dtype, dev if dev.type == "cuda" else None)
        if o is not g and not (isinstance(o, torch.Tensor) and o.dtype == g.dtype and o.shape == g.shape
                               and o.device == dev and o.is_contiguous()):
            check(o, f"out[{i}]", g.dtype, dev, g.shape)
        flat += (g.data_ptr(), o.data_ptr(), g.numel(), TYPES[g.dtype])
    array = (GradTensor * max(1, len(grads))).from_buffer((c_uint64 * max(4, len(flat)))(*flat))
    return array, len(grads), dev


def grad_norm_workspace(count: int) -> int:
    """Bytes of workspace grad_norm and clip_grad_norm take for so many tensors."""
    n = int(load_library().grad_norm_workspace(count))
    if n < 0:
        raise ValueError(f"invalid number of tensors {count}")
    return n


def _run(name, grads, out, norm, workspace, stream, *more):
    lib = load_library()
    array, count, dev = _tensors(grads, out, norm)
    with on_device(dev, stream):
        norm = given_or_new(norm, "norm", F32, dev, ())
        at, size, keep = space(grad_norm_workspace(count), workspace, dev)
        _check(name, getattr(lib, name)(array, count, *more, norm.data_ptr(), at, size, stream_ptr(dev, stream)))
    return norm


def grad_norm(grads, norm=None, workspace=None, stream=None):
    """norm [] (float32, on the GPU) = sqrt(sum over all of ``grads`` of g^2) (see
    include/grad_norm.h).  The gradients are contiguous float32, bfloat16 or float16 tensors
    of one GPU, any number of any shapes.  The workspace is allocated here unless given."""
    return _run("grad_norm", grads, None, norm, workspace, stream)


def clip_grad_norm(grads, max_norm: float, out=None, norm=None, workspace=None, stream=None):
    """norm [] as grad_norm's, of the gradients as they were given; each becomes
    g * min(1, max_norm / (norm + 1e-6)), where it is or in the tensor of ``out`` (one
    for each, of its type and shape) at its place.  Nothing is read back to the host.
    Where the norm is NaN all outputs are, where it is infinite the factor is 0 (and 1 with
    an infinite ``max_norm``, which clips nothing)."""
    if not max_norm >= 0:
        raise ValueError(f"max_norm must be at least 0, got {max_norm}")
    return _run("clip_grad_norm", grads, out, norm, workspace, stream, float(max_norm))
