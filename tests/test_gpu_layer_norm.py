"""The layer norm on the GPU against its formula in float64.

Tolerances.  y and grad_x are 32-bit results rounded once: half a step of the value, and the
arithmetic's own error.  A row's sums are trees of at most 10 + log2(width) additions, half a
2^-24 each, of their terms' magnitudes; a difference to the mean has the mean's error, so what
a value's error is relative to is the row's mean magnitude and its own: 64 roundings of 2^-24
of that.  The variance's error from the mean's is of second order (the differences sum to
nothing).  The weights' gradients are 64-bit sums of products rounded three times, rounded
twice more: 8 roundings of the terms' magnitudes."""
import numpy as np
import pytest

import sequence_reference as R
from parity_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ULP = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


def near(name, got, want, size, ulps):
    half = torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -149
    got = got.double()
    bad = ~((got - want).abs() <= half * want.abs() + ulps * ULP * size + tiny)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {(got - want).abs().max():.3e}"


def make(seed, kind, rows, width, residual, offset=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = TYPES[kind]
    x, w, b = (n(rows, width) + offset).to(t), (1 + 0.3 * n(width)).to(t), n(width).to(t)
    return x, w, b, {"none": None, "same": n(rows, width).to(t), "fp32": n(rows, width)}[residual]


def formula(x, w, b, r):
    h = x.double() if r is None else (x.float() + r.float()).to(r.dtype).double()
    mean = h.mean(-1)
    rstd = 1 / torch.sqrt((h - mean[:, None]).square().mean(-1) + EPS)
    y = (h - mean[:, None]) * rstd[:, None] * w.double() + (0 if b is None else b.double())
    size = (h.abs() + h.abs().mean(-1, keepdim=True)) * rstd[:, None] * w.double().abs() + (0 if b is None else b.double().abs())
    return y, h, mean, rstd, size


SIZES = [(1, 1), (3, 7), (17, 16), (5, 127), (1000, 128), (33, 129), (9, 512), (7, 513), (20, 1000), (3, 2048),
         (2, 2049), (5, 4096), (3, 4101), (2, 8192), (1, 8193), (2, 16384), (600, 33), (5000, 64),
         (9001, 600), (2100, 1500)]  # the last two: more rows than a launch has workgroups


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,width", SIZES)
def test_forward(gpu, kind, rows, width):
    for residual, bias in (("none", True), ("same", False), ("fp32", True)):
        say(f"[layer norm] forward {kind} {rows} {width} {residual}")
        x, w, b, r = make(rows + width, kind, rows, width, residual, offset=0.5)
        b = b if bias else None
        y, h, mean, rstd = gpu.layer_norm_forward(x, w, b, EPS, residual=r)
        want, wh, wm, wr, size = formula(x, w, b, r)
        assert y.dtype == x.dtype and h.dtype == (x.dtype if r is None else r.dtype)
        assert torch.equal(h.double(), wh)
        near("mean", mean, wm, wh.abs().mean(-1), 64)
        if width > 1:
            near("rstd", rstd, wr, wr, 64)
        near("y", y, want, size, 64)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,width", SIZES)
def test_backward(gpu, kind, rows, width):
    for residual, stream in (("same", True), ("fp32", True), ("same", False)):
        say(f"[layer norm] backward {kind} {rows} {width} {residual} {stream}")
        x, w, b, r = make(rows + width + 2, kind, rows, width, residual)
        gy, _, _, gh = make(rows + width + 3, kind, rows, width, residual)
        _, h, mean, rstd = gpu.layer_norm_forward(x, w, b, EPS, residual=r)
        gx, gw, gb = gpu.layer_norm_backward(gy, h, w, mean, rstd, grad_h=gh if stream else None)
        assert gx.dtype == r.dtype and gw.dtype == gb.dtype == torch.float32
        rs = rstd.double()[:, None]
        n = (h.double() - mean.double()[:, None]) * rs
        d = gy.double() * w.double()
        want = rs * (d - d.mean(-1, keepdim=True) - n * (d * n).mean(-1, keepdim=True))
        size = rs * (d.abs() + d.abs().mean(-1, keepdim=True) + n.abs() * (d * n).abs().mean(-1, keepdim=True))
        if stream:
            want, size = want + gh.double(), size + gh.double().abs()
        near("x", gx, want, size, 64)
        near("weight", gw, (gy.double() * n).sum(0), (gy.double() * n).abs().sum(0), 8)
        near("bias", gb, gy.double().sum(0), gy.double().abs().sum(0), 8)


def test_the_formula_is_the_references():
    gen = np.random.default_rng(1)
    h, w, b, gy = (gen.standard_normal(s) for s in ((6, 50), 50, 50, (6, 50)))
    t = lambda a: torch.from_numpy(a)  # noqa: E731
    y, _, mean, rstd, _ = formula(t(h), t(w), t(b), None)
    want = R.layer_norm(h, w, b, EPS)
    for got, ref in zip((y, mean, rstd), want):
        np.testing.assert_allclose(got.numpy(), ref, rtol=1e-13, atol=1e-13)


def test_gradients_against_the_references(gpu):
    """In fp32, where the reference's own adjoint (held to differences) says what is right."""
    gen = np.random.default_rng(2)
    h, w, b, gy = (torch.from_numpy(gen.standard_normal(s)).float() for s in ((40, 300), 300, 300, (40, 300)))
    _, _, mean, rstd = gpu.layer_norm_forward(h.cuda(), w.cuda(), b.cuda(), EPS)
    got = gpu.layer_norm_backward(gy.cuda(), h.cuda(), w.cuda(), mean, rstd)
    h64, w64, b64, g64 = (v.double().numpy() for v in (h, w, b, gy))
    _, m, r = R.layer_norm(h64, w64, b64, EPS)
    for name, t, want in zip(("x", "weight", "bias"), got, R.layer_norm_backward(g64, h64, w64, m, r)):
        # rstd's and the mean's own errors come on top: 128 roundings of the largest magnitude of a sum's terms
        room = 128 * ULP * np.abs(want).max() * (8 if name == "x" else 40)
        assert np.abs(t.double().cpu().numpy() - want).max() <= room, name


def test_rows_far_from_zero_keep_their_variance(gpu):
    """The mean is a thousand times the deviation: differences are exact to 2^-24 of the value,
    6e-5 of the deviation, and the mean's own error shifts them all alike."""
    x, w, b, _ = make(4, "fp32", 50, 1000, "none", offset=1000.0)
    y, h, mean, rstd = gpu.layer_norm_forward(x, w, b, EPS)
    want, _, wm, wr, size = formula(x, w, b, None)
    near("rstd", rstd, wr, wr, 64)
    near("y", y, want, size, 64)


def test_any_address_and_given_buffers(gpu):
    for kind in ("bf16", "fp32"):
        for width in (33, 64, 1500):
            x, w, b, r = make(6, kind, 20, width, "same")
            want = gpu.layer_norm_forward(x, w, b, EPS, residual=r)
            at = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)  # noqa: E731  an element further on
            res = at(r)
            y = at(torch.zeros_like(x))
            got = gpu.layer_norm_forward(at(x), at(w), at(b), EPS, residual=res, h=res, y=y)
            assert got[0] is y and got[1] is res and all(torch.equal(u, v) for u, v in zip(want, got))
            gy = torch.randn_like(x)
            back = gpu.layer_norm_backward(gy, want[1], w, want[2], want[3], grad_h=r)
            gh = at(r)
            got = gpu.layer_norm_backward(at(gy), at(want[1]), at(w), want[2], want[3], grad_h=gh, grad_x=gh)
            assert got[0] is gh and all(torch.equal(u, v) for u, v in zip(back, got))
            none = gpu.layer_norm_backward(gy, want[1], w, want[2], want[3], grad_h=r, want_bias=False)
            assert none[2] is None and torch.equal(none[1], back[1])


def test_no_rows(gpu):
    x, w, b, _ = make(7, "bf16", 0, 24, "none")
    y, h, mean, rstd = gpu.layer_norm_forward(x, w, b, EPS)
    gx, gw, gb = gpu.layer_norm_backward(y, h, w, mean, rstd)
    assert gx.shape == (0, 24) and (gw == 0).all() and (gb == 0).all()


def test_values_that_are_not_finite_stay_in_their_row(gpu):
    for width in (100, 600, 4096):
        x, w, b, r = make(5, "bf16", 6, width, "same")
        want = gpu.layer_norm_forward(x, w, b, EPS, residual=r)
        x[2, 3], x[4, 1] = float("nan"), float("inf")
        got = gpu.layer_norm_forward(x, w, b, EPS, residual=r)
        keep = [0, 1, 3, 5]
        assert all(torch.equal(u[keep], v[keep]) for u, v in zip(want, got))
        assert torch.isnan(got[0][2]).all() and torch.isnan(got[0][4]).all()


def test_equal_bits_on_another_stream_and_replayed(gpu):
    x, w, b, r = make(8, "bf16", 3000, 520, "fp32")
    gy = torch.randn_like(x)

    def work():
        y, h, mean, rstd = gpu.layer_norm_forward(x, w, b, EPS, residual=r)
        return (y, h, mean, rstd, *gpu.layer_norm_backward(gy, h, w, mean, rstd, grad_h=r))

    want = work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = work()
    here = work()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) and torch.equal(u, o) for u, v, o in zip(want, got, here))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    start = x.clone()
    for i in range(3):
        x.copy_(start * (i + 1))
        eager = [t.clone() for t in work()]
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(eager, held))
