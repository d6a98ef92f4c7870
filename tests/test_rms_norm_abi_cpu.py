"""The root-mean-square norm's C ABI and binding without a GPU: exports,
workspace sizes and every refusal, before the HIP runtime is touched."""
import os

import pytest

import cfc_recurrent_cell_amd as C
from cfc_recurrent_cell_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libcfc_amd.so not built (run __graft_entry__.build())")
HEADER = os.path.join(os.path.dirname(_lib.HEADER), "rms_norm.h")
M = 1 << 20
X, R, W, Y, H, RSTD, SC, GH, GX, GW, WS = (0x10000000 + 16 * M * i for i in range(11))
BF16, F16, F32 = _lib.CFC_TYPE_BF16, _lib.CFC_TYPE_F16, _lib.CFC_TYPE_F32
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    return C.load_library()


def fwd(lib, kind=BF16, stream=BF16, rows=64, width=64, x=X, r=R, w=W, eps=1e-6, y=Y, h=H, rstd=RSTD):
    return lib.rms_norm_forward(kind, stream, rows, width, x, r, w, eps, y, h, rstd, None)


def e4(lib, kind=BF16, stream=BF16, rows=64, width=64, x=X, r=R, w=W, eps=1e-6, group=32, y=Y, scales=SC, h=H, rstd=RSTD):
    return lib.rms_norm_forward_e4m3(kind, stream, rows, width, x, r, w, eps, group, y, scales, h, rstd, None)


def bwd(lib, kind=BF16, stream=BF16, rows=64, width=64, gy=Y, h=H, w=W, rstd=RSTD, gh=GH, gx=GX, gw=GW, ws=WS,
        size=1 << 30):
    return lib.rms_norm_backward(kind, stream, rows, width, gy, h, w, rstd, gh, gx, gw, ws, size, None)


def test_exports_every_declared_symbol(lib):
    names = _lib.declared_symbols(HEADER)
    assert set(names) == {"rms_norm_forward", "rms_norm_forward_e4m3", "rms_norm_backward",
                          "rms_norm_backward_workspace"}
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("bad,code", [
    (dict(kind=3), C.CFC_ERR_UNSUPPORTED), (dict(kind=F16), C.CFC_ERR_UNSUPPORTED),
    (dict(kind=F32), C.CFC_ERR_UNSUPPORTED), (dict(rows=-1), C.CFC_ERR_DIM), (dict(width=0), C.CFC_ERR_DIM),
    (dict(width=16385), C.CFC_ERR_UNSUPPORTED), (dict(rows=2 ** 62), C.CFC_ERR_DIM), (dict(w=None), C.CFC_ERR_NULL),
])
def test_sizes_and_types_that_are_refused(lib, bad, code):
    assert fwd(lib, **bad) == code
    assert e4(lib, **bad) == code
    assert bwd(lib, **bad) == code


def test_forward_refusals(lib):
    for f in (fwd, e4):
        assert f(lib, eps=NAN) == C.CFC_ERR_DT
        assert f(lib, eps=-1e-6) == C.CFC_ERR_DT
        assert f(lib, x=None) == C.CFC_ERR_NULL
        assert f(lib, y=None) == C.CFC_ERR_NULL
        assert f(lib, r=None) == C.CFC_ERR_DIM                  # h without a residual
        assert f(lib, r=None, h=None, stream=F32) == C.CFC_ERR_DIM
        for at in (X, R, W, H, RSTD):
            assert f(lib, y=at + 16) == C.CFC_ERR_OVERLAP
        for at in (X, R):
            assert f(lib, h=at + 16) == C.CFC_ERR_OVERLAP        # over it, but not it
        assert f(lib, stream=F32, h=X) == C.CFC_ERR_OVERLAP
        assert f(lib, rstd=X) == C.CFC_ERR_OVERLAP
        assert f(lib, rows=0, x=None, y=None) == C.CFC_OK
    assert e4(lib, scales=None) == C.CFC_ERR_NULL
    assert e4(lib, scales=Y) == C.CFC_ERR_OVERLAP
    for group in (-16, 1, 8, 24, 48, 1024):
        assert e4(lib, group=group) == C.CFC_ERR_DIM


def test_backward_refusals(lib):
    for n in ("gy", "h", "w", "rstd", "gx", "gw", "ws"):
        assert bwd(lib, **{n: None}) == C.CFC_ERR_NULL, n
    need = lib.rms_norm_backward_workspace(64, 64)
    assert need == 4 * 64 * 4  # sixteen rows are one workgroup's
    assert bwd(lib, size=need - 1) == C.CFC_ERR_DIM
    assert bwd(lib, ws=WS + 8) == C.CFC_ERR_DIM
    for at in (Y, H, W, RSTD, GH):
        assert bwd(lib, gx=at + 16) == C.CFC_ERR_OVERLAP
        assert bwd(lib, gw=at) == C.CFC_ERR_OVERLAP
        assert bwd(lib, ws=at) == C.CFC_ERR_OVERLAP
    assert bwd(lib, gw=GX) == C.CFC_ERR_OVERLAP
    assert lib.rms_norm_backward_workspace(-1, 64) == -1
    assert lib.rms_norm_backward_workspace(4, 0) == -1
    assert lib.rms_norm_backward_workspace(4, 16385) == -1


def test_binding_refuses_what_does_not_fit():
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="on a GPU"):
        C.rms_norm_forward(x, x[0], 1e-6)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        C.rms_norm_forward(x.double(), x[0].double(), 1e-6)
    with pytest.raises(ValueError, match="on a GPU"):
        C.rms_norm_backward(x, x, x[0], x[:, 0])
    with pytest.raises(ValueError, match="width"):
        C.rms_norm_backward_workspace(4, 20000)
