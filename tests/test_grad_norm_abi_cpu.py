"""The gradients' norm and clipping, C ABI and binding without a GPU: exports, workspace
sizes and every refusal, before the HIP runtime is touched."""
import os

import pytest

import cfc_recurrent_cell_amd as C
from cfc_recurrent_cell_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libcfc_amd.so not built (run __graft_entry__.build())")
HEADER = os.path.join(os.path.dirname(_lib.HEADER), "grad_norm.h")
M = 1 << 20
G, O, NORM, WS = (0x10000000 + 64 * M * i for i in range(4))
BF16, F32 = _lib.CFC_TYPE_BF16, _lib.CFC_TYPE_F32
NEED = (2048 + 2) * 8


@pytest.fixture(scope="module")
def lib():
    return C.load_library()


def call(lib, tensors, clip=True, count=None, max_norm=1.0, norm=NORM, ws=WS, size=1 << 30):
    array = (_lib.GradTensor * max(1, len(tensors)))(*tensors)
    count = len(tensors) if count is None else count
    if clip:
        return lib.clip_grad_norm(array, count, max_norm, norm, ws, size, None)
    return lib.grad_norm(array, count, norm, ws, size, None)


ONE = (G, O, 100, F32)


def test_exports_every_declared_symbol(lib):
    names = _lib.declared_symbols(HEADER)
    assert set(names) == {"grad_norm", "clip_grad_norm", "grad_norm_workspace"}
    for n in names:
        assert hasattr(lib, n), n


def test_workspace(lib):
    assert lib.grad_norm_workspace(-1) == -1
    assert lib.grad_norm_workspace(0) == 16
    assert lib.grad_norm_workspace(1) == lib.grad_norm_workspace(112) == NEED
    assert lib.grad_norm_workspace(113) == NEED + 2048 * 8
    for clip in (True, False):
        assert call(lib, [ONE], clip, size=NEED - 1) == call(lib, [ONE], clip, ws=WS + 8) == C.CFC_ERR_DIM
        assert call(lib, [ONE], clip, ws=None) == call(lib, [ONE], clip, norm=None) == C.CFC_ERR_NULL
        assert call(lib, [ONE], clip, norm=NORM + 2) == call(lib, [ONE], clip, count=-1) == C.CFC_ERR_DIM
    assert lib.grad_norm(None, 1, NORM, WS, 1 << 30, None) == C.CFC_ERR_NULL


def test_tensors_that_are_refused(lib):
    for clip in (True, False):
        assert call(lib, [ONE, (G + M, O + M, 5, 7)], clip) == C.CFC_ERR_UNSUPPORTED
        assert call(lib, [(G, O, -1, F32)], clip) == call(lib, [(G, O, 1 << 60, F32)], clip) == C.CFC_ERR_DIM
        assert call(lib, [(None, O, 1, F32)], clip) == C.CFC_ERR_NULL
        assert call(lib, [(G + 2, O, 1, F32)], clip) == C.CFC_ERR_DIM
        assert call(lib, [(G, O, 100, F32)], clip, norm=G + 4) == C.CFC_ERR_OVERLAP
        assert call(lib, [(G, O, 100, F32)], clip, ws=G) == C.CFC_ERR_OVERLAP
    assert call(lib, [(G, None, 1, F32)]) == C.CFC_ERR_NULL
    assert call(lib, [(G, O + 1, 1, BF16)]) == C.CFC_ERR_DIM
    for bad in (float("nan"), -1.0, float("-inf")):
        assert call(lib, [ONE], max_norm=bad) == C.CFC_ERR_DT


def test_outputs_that_overlap(lib):
    big = (G, G, 1000, F32)
    for others in ([(G, G, 1000, F32)], [(G + M, G, 10, F32)], [(G + 400, O, 10, F32)], [(G + 400, G + 400, 1, F32)],
                   [(G, O, 1000, F32)], [(G, O, 10, F32)]):
        assert call(lib, [big, *others]) == C.CFC_ERR_OVERLAP
        assert call(lib, [*others, big]) == C.CFC_ERR_OVERLAP
    assert call(lib, [(G, G + 4, 1000, F32)]) == C.CFC_ERR_OVERLAP   # over its own, but not it
    assert call(lib, [(G, O, 1000, F32), (G, O + 2000, 1000, F32)]) == C.CFC_ERR_OVERLAP
    assert call(lib, [(G, O, 100, F32), (G, O + M, 100, F32), (G + 8, O + 16, 4, F32)]) == C.CFC_ERR_OVERLAP
    assert call(lib, [(G, WS, 10, F32)]) == call(lib, [(G, NORM, 10, F32)]) == C.CFC_ERR_OVERLAP


def test_binding_refuses_what_does_not_fit():
    import torch
    x = torch.zeros(4)
    with pytest.raises(TypeError, match="list"):
        C.grad_norm(x)
    with pytest.raises(ValueError, match="on a GPU"):
        C.grad_norm([x])
    with pytest.raises(ValueError, match="at least one"):
        C.grad_norm([])
    with pytest.raises(TypeError, match="torch.Tensor"):
        C.grad_norm([None])
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        C.grad_norm([x.double()])
    with pytest.raises(ValueError, match="out has 0"):
        C.clip_grad_norm([x], 1.0, out=[])
    for bad in (-1.0, float("nan")):
        with pytest.raises(ValueError, match="max_norm"):
            C.clip_grad_norm([x], bad)
    with pytest.raises(ValueError, match="number of tensors"):
        C.grad_norm_workspace(-1)
