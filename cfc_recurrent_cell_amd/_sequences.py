"""How the bindings of the convolution and the scan read a call's sequences of tokens."""
from __future__ import annotations

import torch

from ._delta_rule import _ints
from ._tensors import check, given_or_new


def lead_of(x, offsets, tail: int = 1) -> int:
    """The number of x's leading axes that number its tokens, x [*lead, <tail axes>]."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    lead = 2 if offsets is None else 1
    if x.dim() != lead + tail:
        axes = "[tokens, channels] with offsets" if lead == 1 else "[batch, tokens, channels] without offsets"
        raise ValueError(f"x must be {axes}, got {x.dim()} dimensions")
    return lead


def row_stride(t, name, lead, dtype, device, shape):
    """Elements from one token of t to the next, tokens numbered along its leading axes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor on {device} (got {t.dtype}, {t.device})"
                         if device.type == "cuda" else f"{name} must be a tensor on a GPU (got {t.device})")
    n = t.shape
    if n != shape:
        raise ValueError(f"{name} has shape {tuple(n)}, expected {tuple(shape)}")
    st = t.stride()
    if st[-1] != 1 and n[-1] > 1 and t.numel():
        raise ValueError(f"{name}'s last axis must be dense (its stride is {st[-1]})")
    if lead == 1:
        return st[0]
    if n[1] == 1:
        return st[0]
    if st[0] != n[1] * st[1] and n[0] > 1 and t.numel():
        raise ValueError(f"{name}'s sequences must lie one behind the other (strides {st}): make it contiguous")
    return st[1]


def sequences_of(x, lead, offsets):
    """(sequences, tokens of each or 0, tokens, pointer of the offsets or None).  Rows of a
    step, x [batch, ...] without offsets, are no sequences."""
    n = x.shape
    if offsets is None and lead == 1:
        return 0, 0, n[0], None
    if offsets is None:
        _ints(n[0], n[1])
        return n[0], n[1], n[0] * n[1], None
    check(offsets, "offsets", torch.int32, x.device)
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets must be a vector of the sequences' beginnings and the last one's end")
    _ints(offsets.numel())
    return offsets.numel() - 1, 0, n[0], offsets.data_ptr()


def slots_of(slots, rows, states, shape, dtype, device):
    """The pool's size, after the checks of a pool of states [pool, *shape] and the rows' slots."""
    if not isinstance(states, torch.Tensor) or states.dim() != len(shape) + 1:
        raise ValueError(f"states must be a tensor of {len(shape) + 1} dimensions, a pool of states {tuple(shape)}")
    pool = states.shape[0]
    _ints(pool)
    check(states, "states", dtype, device, (pool, *shape))
    if slots is not None:
        check(slots, "slots", torch.int32, device, (rows,))
    elif pool < rows:
        raise ValueError(f"{rows} rows need as many states, got {pool}")
    return pool


def given_or_cleared(s, bit, t, name, dtype, device, shape):
    """The given buffer of token rows after its checks, or a new one.  Rows behind the last
    packed sequence keep what a given buffer holds; in a new one the call clears them
    (its bit of ``s.clear_rest``), so that what follows over all rows meets no stale memory."""
    if t is not None:
        return check(t, name, dtype, device, shape)
    if s.offsets and s.n_seq == 0:
        return torch.zeros(shape, dtype=dtype, device=device)
    s.clear_rest |= bit
    return given_or_new(None, name, dtype, device, shape)
