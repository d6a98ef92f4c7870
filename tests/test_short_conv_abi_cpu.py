"""The short convolution's C ABI and binding without a GPU: exports, workspace sizes and
every refusal, before the HIP runtime is touched."""
import os
from ctypes import byref

import pytest

import cfc_recurrent_cell_amd as C
from cfc_recurrent_cell_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libcfc_amd.so not built (run __graft_entry__.build())")
HEADER = os.path.join(os.path.dirname(_lib.HEADER), "short_conv.h")
M = 1 << 24
NAMES = ("x", "w", "b", "init", "y", "final", "gy", "gfinal", "gx", "gw", "gb", "ginit", "ws", "offsets", "slots")
AT = {n: 0x10000000 + M * i for i, n in enumerate(NAMES)}
SIZE = dict(type=_lib.CFC_TYPE_BF16, n_seq=2, seq_len=50, n_tokens=100, offsets=None, channels=64, width=4, silu=1, clear_rest=0,
            x_stride=64, grad_y_stride=64)


@pytest.fixture(scope="module")
def lib():
    return C.load_library()


def shape(**over):
    return _lib.ShortConvShape(*{**SIZE, **{k: v for k, v in over.items() if k in SIZE}}.values())


def at(over, *names):
    return [over.get(n, AT[n]) for n in names]


def forward(lib, **over):
    return lib.short_conv_forward(byref(shape(**over)), *at(over, "x", "w", "b", "init", "y", "final"), None)


def backward(lib, **over):
    s = shape(**over)
    return lib.short_conv_backward(byref(s), *at(over, "x", "w", "b", "init", "gy", "gfinal", "gx", "gw", "gb", "ginit", "ws"),
                                   over.get("size", lib.short_conv_backward_workspace(byref(s))), None)


def step(lib, **over):
    return lib.short_conv_step(byref(shape(**over)), *at(over, "x", "w", "b", "init"), over.get("pool", 128),
                               *at(over, "slots", "y"), None)


def test_exports_every_declared_symbol(lib):
    names = _lib.declared_symbols(HEADER)
    assert set(names) == {"short_conv_forward", "short_conv_backward", "short_conv_backward_workspace", "short_conv_step"}
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("bad,code", [
    (dict(type=-1), C.CFC_ERR_UNSUPPORTED), (dict(channels=0), C.CFC_ERR_DIM), (dict(width=0), C.CFC_ERR_DIM),
    (dict(width=1), C.CFC_ERR_UNSUPPORTED), (dict(width=5), C.CFC_ERR_UNSUPPORTED), (dict(x_stride=-1), C.CFC_ERR_DIM),
    (dict(grad_y_stride=-1), C.CFC_ERR_DIM), (dict(n_tokens=-1), C.CFC_ERR_DIM), (dict(n_tokens=1 << 31), C.CFC_ERR_UNSUPPORTED),
    (dict(channels=1 << 30), C.CFC_ERR_UNSUPPORTED), (dict(x_stride=1 << 62), C.CFC_ERR_DIM)])
def test_shapes_that_are_refused(lib, bad, code):
    assert forward(lib, **bad) == backward(lib, **bad) == step(lib, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(n_seq=-1), C.CFC_ERR_DIM), (dict(seq_len=49), C.CFC_ERR_DIM), (dict(seq_len=-1), C.CFC_ERR_DIM),
    (dict(n_seq=(1 << 31) - 1, offsets=AT["offsets"]), C.CFC_ERR_UNSUPPORTED)])
def test_sequences_that_are_refused(lib, bad, code):
    assert forward(lib, **bad) == backward(lib, **bad, size=1 << 40) == code
    assert lib.short_conv_backward_workspace(byref(shape(**bad))) == -1


def test_null_arguments_and_workspace(lib):
    assert lib.short_conv_forward(None, *[None] * 7) == C.CFC_ERR_NULL
    for n in ("x", "w", "y"):
        assert forward(lib, **{n: None}) == step(lib, **{n: None}) == C.CFC_ERR_NULL, n
    assert step(lib, init=None) == C.CFC_ERR_NULL
    for n in ("x", "w", "gy", "gx", "gw", "ws"):
        assert backward(lib, **{n: None}) == C.CFC_ERR_NULL, n
    need = lib.short_conv_backward_workspace(byref(shape()))
    assert need == 7 * 5 * 64 * 4  # seven groups of 16 tokens
    assert backward(lib, size=need - 1) == C.CFC_ERR_DIM
    assert backward(lib, ws=AT["ws"] + 8) == C.CFC_ERR_DIM


def test_addresses(lib):
    for n in ("x", "w", "b", "init", "y", "final"):
        assert forward(lib, **{n: AT[n] + 1}) == C.CFC_ERR_DIM, n
    for n in ("x", "w", "b"):
        assert forward(lib, y=AT[n] + 2) == C.CFC_ERR_OVERLAP, n
        assert forward(lib, final=AT[n]) == C.CFC_ERR_OVERLAP, n
        assert step(lib, y=AT[n]) == step(lib, init=AT[n]) == C.CFC_ERR_OVERLAP, n
    for n in ("x", "w", "b", "init", "gy", "gfinal"):
        assert backward(lib, gx=AT[n]) == backward(lib, ginit=AT[n]) == backward(lib, ws=AT[n]) == C.CFC_ERR_OVERLAP, n
    assert forward(lib, final=AT["init"] + 2) == C.CFC_ERR_OVERLAP
    assert forward(lib, final=AT["init"], y=AT["init"]) == C.CFC_ERR_OVERLAP
    assert forward(lib, offsets=AT["y"]) == step(lib, slots=AT["y"]) == C.CFC_ERR_OVERLAP
    assert backward(lib, gw=AT["gb"]) == C.CFC_ERR_OVERLAP


def test_step_refusals_and_nothing_to_do(lib):
    assert step(lib, pool=-1) == step(lib, slots=None, pool=99) == C.CFC_ERR_DIM
    assert step(lib, n_tokens=0, x=None, y=None) == C.CFC_OK
    assert forward(lib, n_seq=0, n_tokens=0, x=None) == C.CFC_OK


def test_binding_refuses_what_does_not_fit():
    import torch
    x, w = torch.zeros(2, 3, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="on a GPU"):
        C.short_conv_forward(x, w)
    with pytest.raises(ValueError, match="without offsets"):
        C.short_conv_forward(x[0], w)
    with pytest.raises(ValueError, match="with offsets"):
        C.short_conv_forward(x, w, offsets=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        C.short_conv_backward(x.double(), w, x)
    with pytest.raises(ValueError, match="batch, channels"):
        C.short_conv_step(x, w, x)
