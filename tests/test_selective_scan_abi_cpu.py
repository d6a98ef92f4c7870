"""The selective scan's C ABI and binding without a GPU: exports, workspace sizes and every
refusal, before the HIP runtime is touched."""
import os
from ctypes import byref

import pytest

import cfc_recurrent_cell_amd as C
from cfc_recurrent_cell_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libcfc_amd.so not built (run __graft_entry__.build())")
HEADER = os.path.join(os.path.dirname(_lib.HEADER), "selective_scan.h")
M = 1 << 24
NAMES = ("x", "dt", "a", "b", "c", "d", "z", "bias", "init", "y", "final", "gy", "gfinal", "gx", "gdt", "ga", "gb", "gc", "gd",
         "gz", "gbias", "ginit", "ws", "offsets", "slots")
AT = {n: 0x10000000 + M * i for i, n in enumerate(NAMES)}
SIZE = dict(type=_lib.CFC_TYPE_BF16, n_seq=2, seq_len=50, n_tokens=100, offsets=None, channels=64, groups=2, state=16, softplus=1,
            clear_rest=0, x_stride=64, dt_stride=64, z_stride=64, grad_y_stride=64, b_stride_t=32, b_stride_g=16, c_stride_t=32,
            c_stride_g=16)


@pytest.fixture(scope="module")
def lib():
    return C.load_library()


def shape(**over):
    s = {**SIZE, **{k: v for k, v in over.items() if k in SIZE}}
    return _lib.SelectiveScanShape(*s.values())


def at(over, *names):
    return [over.get(n, AT[n]) for n in names]


def forward(lib, **over):
    return lib.selective_scan_forward(byref(shape(**over)), *at(over, "x", "dt", "a", "b", "c", "d", "z", "bias", "init", "y", "final"), None)


def backward(lib, **over):
    s = shape(**over)
    return lib.selective_scan_backward(
        byref(s), *at(over, "x", "dt", "a", "b", "c", "d", "z", "bias", "init", "gy", "gfinal", "gx", "gdt", "ga", "gb", "gc", "gd",
                      "gz", "gbias", "ginit", "ws"), over.get("size", lib.selective_scan_backward_workspace(byref(s))), None)


def step(lib, **over):
    return lib.selective_scan_step(byref(shape(**over)), *at(over, "x", "dt", "a", "b", "c", "d", "z", "bias", "init"),
                                   over.get("pool", 128), *at(over, "slots", "y"), None)


def test_exports_every_declared_symbol(lib):
    names = _lib.declared_symbols(HEADER)
    assert set(names) == {"selective_scan_forward", "selective_scan_backward", "selective_scan_backward_workspace",
                          "selective_scan_step"}
    for n in names:
        assert hasattr(lib, n), n


SHAPES = [(dict(type=3), C.CFC_ERR_UNSUPPORTED), (dict(channels=0), C.CFC_ERR_DIM), (dict(groups=0), C.CFC_ERR_DIM),
          (dict(groups=3), C.CFC_ERR_DIM), (dict(state=0), C.CFC_ERR_DIM), (dict(state=65), C.CFC_ERR_UNSUPPORTED),
          (dict(x_stride=-1), C.CFC_ERR_DIM), (dict(c_stride_g=-1), C.CFC_ERR_DIM), (dict(n_tokens=-1), C.CFC_ERR_DIM),
          (dict(n_tokens=1 << 31), C.CFC_ERR_UNSUPPORTED)]
SEQUENCES = [(dict(n_seq=-1), C.CFC_ERR_DIM), (dict(seq_len=49), C.CFC_ERR_DIM), (dict(seq_len=-1), C.CFC_ERR_DIM),
             (dict(n_seq=(1 << 31) - 1, offsets=AT["offsets"]), C.CFC_ERR_UNSUPPORTED),
             (dict(n_seq=1 << 30, offsets=AT["offsets"]), C.CFC_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("bad,code", SHAPES)
def test_shapes_that_are_refused(lib, bad, code):
    assert forward(lib, **bad) == backward(lib, **bad) == step(lib, **bad) == code


def test_strides_that_are_refused(lib):
    """Of sequences, 64 rows are less than 2^31 bytes, and rows alone anything that has an address."""
    for n in ("x_stride", "dt_stride", "z_stride", "b_stride_t", "c_stride_t"):
        assert step(lib, **{n: 1 << 62}) == C.CFC_ERR_DIM, n
        for stride in (1 << 62, 1 << 24):
            assert forward(lib, **{n: stride}) == backward(lib, **{n: stride}) == C.CFC_ERR_UNSUPPORTED, n
        alone = dict(n_seq=100, seq_len=1)
        assert forward(lib, **alone, **{n: 1 << 62}) == backward(lib, **alone, **{n: 1 << 62}) == C.CFC_ERR_DIM, n
    assert backward(lib, grad_y_stride=1 << 24) == C.CFC_ERR_UNSUPPORTED
    assert forward(lib, channels=1 << 24, groups=1) == step(lib, channels=1 << 24, groups=1) == C.CFC_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad,code", SEQUENCES)
def test_sequences_that_are_refused(lib, bad, code):
    assert forward(lib, **bad) == backward(lib, **bad, size=1 << 40) == code
    assert lib.selective_scan_backward_workspace(byref(shape(**bad))) == -1


def test_null_arguments(lib):
    assert lib.selective_scan_forward(None, *[None] * 12) == C.CFC_ERR_NULL
    for n in ("x", "dt", "a", "b", "c", "y"):
        assert forward(lib, **{n: None}) == C.CFC_ERR_NULL, n
        assert step(lib, **{n: None}) == C.CFC_ERR_NULL, n
    assert step(lib, init=None) == C.CFC_ERR_NULL
    for n in ("x", "dt", "a", "b", "c", "gy", "gx", "gdt", "ga", "gb", "gc", "gz", "ws"):
        assert backward(lib, **{n: None}) == C.CFC_ERR_NULL, n
    assert backward(lib, z=None) == C.CFC_ERR_DIM  # a gradient of z without z


def test_workspace(lib):
    need = lib.selective_scan_backward_workspace(byref(shape()))
    # states before the blocks of 64 tokens (at most 100 / 64 + 2 of them), b's and c's partial sums of two
    # workgroups each, and two rows of a's, d's and dt_bias's
    assert need == 3 * 64 * 16 * 4 + 2 * 2 * 100 * 32 * 4 + 2 * 64 * 18 * 4
    assert backward(lib, size=need - 1) == C.CFC_ERR_DIM
    assert backward(lib, ws=AT["ws"] + 8) == C.CFC_ERR_DIM
    huge = dict(n_seq=1, seq_len=1 << 30, n_tokens=1 << 30)
    assert lib.selective_scan_backward_workspace(byref(shape(**huge))) == -1


def test_addresses(lib):
    for n in ("x", "dt", "a", "b", "c", "d", "z", "bias", "init", "y", "final"):
        assert forward(lib, **{n: AT[n] + 1}) == C.CFC_ERR_DIM, n
    for n in ("x", "dt", "a", "b", "c", "d", "z", "bias"):
        assert forward(lib, y=AT[n] + 2) == C.CFC_ERR_OVERLAP, n
        assert forward(lib, final=AT[n]) == C.CFC_ERR_OVERLAP, n
        assert step(lib, y=AT[n]) == C.CFC_ERR_OVERLAP, n
        assert step(lib, init=AT[n]) == C.CFC_ERR_OVERLAP, n
        assert backward(lib, gx=AT[n]) == C.CFC_ERR_OVERLAP, n
        assert backward(lib, ws=AT[n]) == C.CFC_ERR_OVERLAP, n
    assert forward(lib, final=AT["init"] + 4) == C.CFC_ERR_OVERLAP
    assert forward(lib, final=AT["init"], y=AT["init"]) == C.CFC_ERR_OVERLAP
    assert forward(lib, offsets=AT["y"]) == C.CFC_ERR_OVERLAP
    assert step(lib, slots=AT["y"]) == C.CFC_ERR_OVERLAP
    assert backward(lib, ginit=AT["gfinal"] + 4) == C.CFC_ERR_OVERLAP
    assert backward(lib, ginit=AT["gfinal"], gx=AT["gfinal"]) == C.CFC_ERR_OVERLAP
    assert backward(lib, gx=AT["gdt"]) == C.CFC_ERR_OVERLAP
    assert backward(lib, gd=AT["ws"]) == C.CFC_ERR_OVERLAP


def test_step_refusals_and_nothing_to_do(lib):
    assert step(lib, pool=-1) == C.CFC_ERR_DIM
    assert step(lib, slots=None, pool=99) == C.CFC_ERR_DIM
    assert step(lib, n_tokens=0, x=None, y=None) == C.CFC_OK
    assert forward(lib, n_seq=0, n_tokens=0, x=None) == C.CFC_OK


def test_binding_refuses_what_does_not_fit():
    import torch
    x, a, b = torch.zeros(2, 3, 8), torch.zeros(8, 4), torch.zeros(2, 3, 1, 4)
    with pytest.raises(ValueError, match="on a GPU"):
        C.selective_scan_forward(x, x, a, b, b)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        C.selective_scan_forward(x.double(), x, a, b, b)
    with pytest.raises(ValueError, match="without offsets"):
        C.selective_scan_forward(x[0], x[0], a, b[0], b[0])
    with pytest.raises(ValueError, match="with offsets"):
        C.selective_scan_forward(x, x, a, b, b, offsets=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="torch.Tensor"):
        C.selective_scan_forward([1], x, a, b, b)
    with pytest.raises(ValueError, match="batch, channels"):
        C.selective_scan_step(x, x, a, b, b, a)
    with pytest.raises(ValueError, match="on a GPU"):
        C.selective_scan_backward(x, x, a, b, b, x)
