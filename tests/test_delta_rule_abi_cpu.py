"""The gated delta rule's C ABI and binding without a GPU: exports, workspace
sizes and every refusal.  Each call here fails its checks (or has nothing to
do) before the HIP runtime is touched."""
import ctypes
import os

import pytest

import cfc_recurrent_cell_amd as C
from cfc_recurrent_cell_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libcfc_amd.so not built (run __graft_entry__.build())")
HEADER = os.path.join(os.path.dirname(_lib.HEADER), "delta_rule.h")
M = 1 << 20
Q, K, V, G, BETA, S0, O, S1, WS, GO = (0x10000000 + 16 * M * i for i in range(10))
GRADS = [0x30000000 + 16 * M * i for i in range(6)]
BF16, F16, F32 = _lib.CFC_TYPE_BF16, _lib.CFC_TYPE_F16, _lib.CFC_TYPE_F32


@pytest.fixture(scope="module")
def lib():
    return C.load_library()


def shape(type=BF16, n_seq=2, seq_len=100, n_tokens=None, offsets=None, hk=2, hv=4, dk=64, dv=32, scale=1.0, **strides):
    s = _lib.DeltaRuleShape(type, n_seq, seq_len, n_seq * seq_len if n_tokens is None else n_tokens, offsets, hk, hv,
                            dk, dv, scale)
    for n, (h, d) in {"q": (hk, dk), "k": (hk, dk), "v": (hv, dv), "go": (hv, dv)}.items():
        setattr(s, n + "_stride_t", strides.get(n + "_t", h * d))
        setattr(s, n + "_stride_h", strides.get(n + "_h", d))
    return s


def fwd(lib, s, q=Q, k=K, v=V, g=G, beta=BETA, s0=S0, o=O, s1=S1, ws=WS, size=1 << 40):
    return lib.delta_rule_forward(ctypes.byref(s) if s is not None else None, q, k, v, g, beta, s0, o, s1, ws, size,
                                  None)


def bwd(lib, s, grads=GRADS, q=Q, s0=S0, go=GO, s1=S1, ws=WS, size=1 << 40):
    return lib.delta_rule_backward(ctypes.byref(s), q, K, V, G, BETA, s0, go, s1, *grads, ws, size, None)


def step(lib, s, q=Q, states=S0, pool=2, slots=None, o=O):
    return lib.delta_rule_step(ctypes.byref(s), q, K, V, G, BETA, states, pool, slots, o, None)


def test_exports_every_declared_symbol(lib):
    names = _lib.declared_symbols(HEADER)
    assert set(names) == {"delta_rule_forward", "delta_rule_backward", "delta_rule_step",
                          "delta_rule_forward_workspace", "delta_rule_backward_workspace"}
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("bad,code", [
    (dict(type=7), C.CFC_ERR_UNSUPPORTED), (dict(n_seq=-1, n_tokens=0), C.CFC_ERR_DIM),
    (dict(seq_len=-1), C.CFC_ERR_DIM), (dict(n_tokens=201), C.CFC_ERR_DIM), (dict(n_tokens=-1), C.CFC_ERR_DIM),
    (dict(n_tokens=2 ** 31, offsets=GRADS[0]), C.CFC_ERR_DIM), (dict(hk=0), C.CFC_ERR_DIM), (dict(hv=3), C.CFC_ERR_DIM),
    (dict(hv=0), C.CFC_ERR_DIM), (dict(dk=0), C.CFC_ERR_DIM), (dict(dv=-4), C.CFC_ERR_DIM),
    (dict(dk=129), C.CFC_ERR_UNSUPPORTED), (dict(dv=257), C.CFC_ERR_UNSUPPORTED),
    (dict(scale=float("nan")), C.CFC_ERR_DT), (dict(scale=float("inf")), C.CFC_ERR_DT),
    (dict(q_t=-1), C.CFC_ERR_DIM), (dict(v_h=-32), C.CFC_ERR_DIM), (dict(go_t=-1), C.CFC_ERR_DIM),
    (dict(hk=1, hv=70000), C.CFC_ERR_UNSUPPORTED), (dict(q_t=2 ** 62), C.CFC_ERR_UNSUPPORTED),
    (dict(n_seq=2 ** 31 - 1, seq_len=0, n_tokens=0), C.CFC_ERR_UNSUPPORTED),
])
def test_shapes_that_are_refused(lib, bad, code):
    s = shape(**bad)
    assert fwd(lib, s) == code
    assert bwd(lib, s) == code
    assert lib.delta_rule_forward_workspace(ctypes.byref(s)) == -1
    assert lib.delta_rule_backward_workspace(ctypes.byref(s)) == -1


def test_null_arguments(lib):
    assert fwd(lib, None) == C.CFC_ERR_NULL
    for n in ("q", "k", "v", "g", "beta", "o", "ws"):
        assert fwd(lib, shape(), **{n: None}) == C.CFC_ERR_NULL, n
    assert bwd(lib, shape(), go=None) == C.CFC_ERR_NULL
    assert bwd(lib, shape(), ws=None) == C.CFC_ERR_NULL
    for i in range(5):
        assert bwd(lib, shape(), grads=[None if j == i else p for j, p in enumerate(GRADS)]) == C.CFC_ERR_NULL
    assert lib.delta_rule_forward_workspace(None) == -1


def test_no_sequences_need_nothing(lib):
    s = shape(n_seq=0)
    assert lib.delta_rule_forward_workspace(ctypes.byref(s)) == 0
    assert fwd(lib, s, q=None, o=None, ws=None, size=0) == C.CFC_OK
    assert bwd(lib, s, ws=None, size=0) == C.CFC_OK
    assert step(lib, shape(n_seq=0), q=None, pool=0, states=None) == C.CFC_OK


def test_workspace_is_checked(lib):
    s = shape()
    for call, size in ((fwd, lib.delta_rule_forward_workspace), (bwd, lib.delta_rule_backward_workspace)):
        need = size(ctypes.byref(s))
        assert need > 0 and need % 16 == 0
        assert call(lib, s, size=need - 1) == C.CFC_ERR_DIM
        assert call(lib, s, ws=WS + 8) == C.CFC_ERR_DIM
        for at in (Q, K, V, G, BETA, S0, S1, Q - need + 16, *((GO, *GRADS) if call is bwd else (O,))):
            assert call(lib, s, ws=at, size=need) == C.CFC_ERR_OVERLAP, hex(at)
    # short sequences take none
    assert lib.delta_rule_forward_workspace(ctypes.byref(shape(seq_len=3))) == 0


def test_overlaps(lib):
    s = shape()
    for at in (Q, K, V, G, BETA, S0, S1):
        assert fwd(lib, s, o=at + 64) == C.CFC_ERR_OVERLAP
    assert fwd(lib, s, s1=S0 + 64) == C.CFC_ERR_OVERLAP       # over it, but not it
    assert fwd(lib, s, o=S0, s1=S0) == C.CFC_ERR_OVERLAP
    # a strided q reaches further than its elements
    assert fwd(lib, shape(q_t=4 * M // 200), o=Q + 2 * M) == C.CFC_ERR_OVERLAP
    for i in range(6):
        for at in (Q, GO, S0, GRADS[(i + 1) % 6]):
            grads = [at + 64 if j == i else p for j, p in enumerate(GRADS)]
            assert bwd(lib, s, grads=grads) == C.CFC_ERR_OVERLAP, (i, hex(at))
    # offsets are an input too
    assert fwd(lib, shape(offsets=O + 64), ) == C.CFC_ERR_OVERLAP


def test_step_refusals(lib):
    s = shape(n_tokens=2)
    assert step(lib, s, pool=1) == C.CFC_ERR_DIM                       # fewer states than rows
    assert step(lib, s, pool=-1, slots=GO) == C.CFC_ERR_DIM
    assert step(lib, s, states=None) == C.CFC_ERR_NULL
    assert step(lib, s, q=None) == C.CFC_ERR_NULL
    assert step(lib, s, o=None) == C.CFC_ERR_NULL
    assert step(lib, s, o=S0 + 64) == C.CFC_ERR_OVERLAP
    assert step(lib, s, o=Q) == C.CFC_ERR_OVERLAP
    assert step(lib, s, states=Q) == C.CFC_ERR_OVERLAP
    assert step(lib, s, slots=S0) == C.CFC_ERR_OVERLAP
    assert step(lib, shape(n_tokens=2, dk=200)) == C.CFC_ERR_UNSUPPORTED


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch
    q = torch.zeros(1, 4, 2, 8)
    g = torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="on a GPU"):
        C.delta_rule_forward(q, q, q, g, g)
    with pytest.raises(ValueError, match="without offsets"):
        C.delta_rule_forward(q[0], q[0], q[0], g[0], g[0])
    with pytest.raises(ValueError, match="with offsets"):
        C.delta_rule_backward(q, q, q, g, g, q, offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="batch, heads, dim"):
        C.delta_rule_step(q, q, q, g, g, torch.zeros(1, 2, 8, 8))


def test_more_chunks_than_a_launch_has(lib):
    """The gradients' last kernel has 512 threads a chunk, and a launch fewer than 2^32."""
    for n, ok in ((1 << 28, True), ((1 << 29) - 64 * 8, True), (1 << 29, False), (3 << 28, False)):
        s = shape(n_seq=1, seq_len=n, hk=1, hv=1, dk=1, dv=1)
        for size in (lib.delta_rule_forward_workspace, lib.delta_rule_backward_workspace):
            assert (size(ctypes.byref(s)) > 0) == ok, n
        if not ok:
            assert fwd(lib, s) == C.CFC_ERR_UNSUPPORTED and bwd(lib, s) == C.CFC_ERR_UNSUPPORTED


def test_a_stream_of_another_device_is_refused():
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace

    from cfc_recurrent_cell_amd._tensors import on_device
    with pytest.raises(ValueError, match="cuda:1"):
        on_device(torch.device("cuda", 0), SimpleNamespace(device=torch.device("cuda", 1)))


@pytest.mark.parametrize("seqs,heads,longest", [(1, 1, 8), (1, 32, 10), (4, 32, 16), (16, 32, 32), (64, 64, 32)])
def test_short_sequences_need_no_workspace(lib, seqs, heads, longest):
    need = [lib.delta_rule_forward_workspace(ctypes.byref(shape(n_seq=seqs, seq_len=n, hk=1, hv=heads)))
            for n in (longest, longest + 1)]
    assert need[0] == 0 < need[1]


def test_row_strides_count_only_where_chunks_have_rows(lib):
    """One-token and few-token slices of a long tensor: rows 2^24 elements (of 64, 2^31 bytes) apart."""
    def needs(**sizes):
        s = shape(hk=16, hv=16, dk=128, dv=128, **{n: 1 << 24 for n in ("q_t", "k_t", "v_t", "go_t")}, **sizes)
        return [f(ctypes.byref(s)) for f in (lib.delta_rule_forward_workspace, lib.delta_rule_backward_workspace)]

    for seqs in (1, 3):
        forward, backward = needs(n_seq=seqs, seq_len=1)
        assert forward == 0 and backward > 0
        assert needs(n_seq=seqs, seq_len=5) == [0, -1]
        assert needs(n_seq=seqs, seq_len=100) == [-1, -1]
    assert needs(n_seq=1, n_tokens=5, offsets=GRADS[0]) == [0, -1]
    assert needs(n_seq=1, n_tokens=100, offsets=GRADS[0]) == [-1, -1]
    s = shape(seq_len=5, k_t=1 << 62)
    assert fwd(lib, s) == C.CFC_ERR_DIM      # the array's end is past 64 bits
    assert bwd(lib, s) == C.CFC_ERR_UNSUPPORTED


def test_the_stride_limit_is_named():
    from cfc_recurrent_cell_amd._delta_rule import _size
    with pytest.raises(ValueError, match="2\\^31 bytes"):
        _size(-1)


def test_sizes_past_32_bits_are_refused():
    from cfc_recurrent_cell_amd._delta_rule import _ints
    _ints(0, 2 ** 31 - 1)
    with pytest.raises(ValueError, match="32 bits"):
        _ints(4, 2 ** 32 + 4)
