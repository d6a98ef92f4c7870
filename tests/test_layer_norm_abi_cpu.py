"""The layer norm's C ABI and binding without a GPU: exports, workspace sizes and every
refusal, before the HIP runtime is touched."""
import os

import pytest

import cfc_recurrent_cell_amd as C
from cfc_recurrent_cell_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libcfc_amd.so not built (run __graft_entry__.build())")
HEADER = os.path.join(os.path.dirname(_lib.HEADER), "layer_norm.h")
M = 1 << 20
X, R, W, B, Y, H, MEAN, RSTD, GH, GX, GW, GB, WS = (0x10000000 + 16 * M * i for i in range(13))
BF16, F16, F32 = _lib.CFC_TYPE_BF16, _lib.CFC_TYPE_F16, _lib.CFC_TYPE_F32


@pytest.fixture(scope="module")
def lib():
    return C.load_library()


def fwd(lib, kind=BF16, stream=BF16, rows=64, width=64, x=X, r=R, w=W, b=B, eps=1e-6, y=Y, h=H, mean=MEAN, rstd=RSTD):
    return lib.layer_norm_forward(kind, stream, rows, width, x, r, w, b, eps, y, h, mean, rstd, None)


def bwd(lib, kind=BF16, stream=BF16, rows=64, width=64, gy=Y, h=H, w=W, mean=MEAN, rstd=RSTD, gh=GH, gx=GX, gw=GW, gb=GB, ws=WS,
        size=1 << 30):
    return lib.layer_norm_backward(kind, stream, rows, width, gy, h, w, mean, rstd, gh, gx, gw, gb, ws, size, None)


def test_exports_every_declared_symbol(lib):
    names = _lib.declared_symbols(HEADER)
    assert set(names) == {"layer_norm_forward", "layer_norm_backward", "layer_norm_backward_workspace"}
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("bad,code", [
    (dict(kind=3), C.CFC_ERR_UNSUPPORTED), (dict(kind=F16), C.CFC_ERR_UNSUPPORTED),
    (dict(kind=F32), C.CFC_ERR_UNSUPPORTED), (dict(rows=-1), C.CFC_ERR_DIM), (dict(width=0), C.CFC_ERR_DIM),
    (dict(width=16385), C.CFC_ERR_UNSUPPORTED), (dict(rows=2 ** 62), C.CFC_ERR_DIM), (dict(w=None), C.CFC_ERR_NULL),
    (dict(w=W + 1), C.CFC_ERR_DIM), (dict(h=H + 1), C.CFC_ERR_DIM), (dict(rstd=RSTD + 2), C.CFC_ERR_DIM)])
def test_what_both_refuse(lib, bad, code):
    assert fwd(lib, **bad) == code
    assert bwd(lib, **bad) == code


def test_forward_refusals(lib):
    assert fwd(lib, eps=float("nan")) == fwd(lib, eps=-1e-6) == C.CFC_ERR_DT
    assert fwd(lib, x=None) == fwd(lib, y=None) == C.CFC_ERR_NULL
    assert fwd(lib, r=None) == fwd(lib, r=None, h=None, stream=F32) == C.CFC_ERR_DIM
    for at in (X, R, W, B, H, MEAN, RSTD):
        assert fwd(lib, y=at + 16) == C.CFC_ERR_OVERLAP
    for at in (X, R):
        assert fwd(lib, h=at + 16) == C.CFC_ERR_OVERLAP  # over it, but not it
    assert fwd(lib, stream=F32, h=X) == C.CFC_ERR_OVERLAP
    assert fwd(lib, mean=RSTD) == C.CFC_ERR_OVERLAP
    assert fwd(lib, rows=0, x=None, y=None) == C.CFC_OK


def test_backward_refusals(lib):
    for n in ("gy", "h", "w", "mean", "rstd", "gx", "gw", "ws"):
        assert bwd(lib, **{n: None}) == C.CFC_ERR_NULL, n
    need = lib.layer_norm_backward_workspace(64, 64)
    assert need == 4 * 64 * 8  # sixteen rows are one workgroup's
    assert bwd(lib, size=need - 1) == bwd(lib, ws=WS + 8) == C.CFC_ERR_DIM
    for at in (Y, H, W, MEAN, RSTD, GH):
        assert bwd(lib, gx=at + 16) == bwd(lib, gw=at) == bwd(lib, gb=at) == bwd(lib, ws=at) == C.CFC_ERR_OVERLAP
    assert bwd(lib, gw=GX) == bwd(lib, gb=GW) == C.CFC_ERR_OVERLAP
    assert lib.layer_norm_backward_workspace(-1, 64) == lib.layer_norm_backward_workspace(4, 0) == -1
    assert lib.layer_norm_backward_workspace(4, 16385) == -1


def test_binding_refuses_what_does_not_fit():
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="on a GPU"):
        C.layer_norm_forward(x, x[0], x[0], 1e-6)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        C.layer_norm_forward(x.double(), x[0].double(), None, 1e-6)
    with pytest.raises(ValueError, match="on a GPU"):
        C.layer_norm_backward(x, x, x[0], x[:, 0], x[:, 0])
    with pytest.raises(ValueError, match="width"):
        C.layer_norm_backward_workspace(4, 20000)
