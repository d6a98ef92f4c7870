"""The root-mean-square norm on the GPU against its formula in float64.

Tolerances.  y and grad_x are 32-bit results rounded once: eps_t / 2 of the
value, and the arithmetic's own error.  rstd is off by the sum of squares'
(a tree of positive terms: at most 10 + log2(width) additions deep, half a
2^-24 each, halved by the root) and by four roundings; y by two more.  A
difference (grad_x) has the error of its largest term, a sum over rows
(grad_weight) that of its terms' magnitudes' sum, with rows / parts + log2 ...
additions: at most 64 roundings of 2^-24 are allowed everywhere below, which
holds for every size here (at most 32 rows for a workgroup's slot).  An e4m3
value is the nearest one or, where a tie is within the arithmetic's error, its
neighbour: off by half a step (2^-4 of the value, or 2^-10 where e4m3 is
subnormal) and that error."""
import numpy as np
import pytest

from parity_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ULP = 64 * 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return torch.device("cuda:0")


def make(seed, kind, rows, width, residual):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = TYPES[kind]
    x, w = n(rows, width).to(t), (1 + 0.3 * n(width)).to(t)
    r = {"none": None, "same": n(rows, width).to(t), "fp32": n(rows, width)}[residual]
    return x, w, r


def formula(x, w, r):
    h = x.double() if r is None else (x.float() + r.float()).to(r.dtype).double()
    rstd = 1 / torch.sqrt(h.square().mean(-1) + EPS)
    return h * rstd[..., None] * w.double(), h, rstd


def near(got, want, half_step, size=None, floor=0.0):
    size = want.abs() if size is None else size
    bad = ~((got.double() - want).abs() <= half_step * want.abs() + ULP * size + floor)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {(got.double() - want).abs().max():.3e}"


def floor_of(t):
    return 2.0 ** -25 if t == torch.float16 else 0.0


SIZES = [(1, 1), (3, 7), (17, 16), (5, 127), (1000, 128), (33, 129), (9, 512), (7, 513), (20, 1000), (3, 2048),
         (2, 2049), (5, 4096), (3, 4104), (2, 8192), (1, 8193), (2, 16384), (600, 33), (5000, 64),
         (9001, 600), (2100, 1500)]  # the last two: more rows than a launch has workgroups


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,width", SIZES)
def test_forward(kind, rows, width):
    import cfc_recurrent_cell_amd as C
    for residual in ("none", "same", "fp32"):
        say(f"[norm] forward {kind} {rows} {width} {residual}")
        x, w, r = make(rows + width, kind, rows, width, residual)
        y, h, rstd = C.rms_norm_forward(x, w, EPS, residual=r)
        want, wh, wr = formula(x, w, r)
        assert y.dtype == x.dtype and h.dtype == (x.dtype if r is None else r.dtype)
        assert torch.equal(h.double(), wh)
        near(rstd, wr, 0.0)
        near(y, want, torch.finfo(x.dtype).eps / 2, floor=floor_of(x.dtype))


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,width", SIZES)
def test_e4m3(kind, rows, width):
    import cfc_recurrent_cell_amd as C
    for residual, group in (("none", 0), ("same", 16), ("fp32", 128), ("same", 512), ("none", 64)):
        say(f"[norm] e4m3 {kind} {rows} {width} {residual} {group}")
        x, w, r = make(rows + width + 1, kind, rows, width, residual)
        y, scales, h = C.rms_norm_forward_e4m3(x, w, EPS, residual=r, group=group)
        want, wh, _ = formula(x, w, r)
        assert torch.equal(h.double(), wh)
        cols = group or width
        for at in range(0, width, cols):
            part = want[:, at:at + cols]
            top = part.abs().amax(-1)
            s = scales[:, at // cols]
            near(s, torch.where(top > 0, top, torch.ones_like(top)) / 448, 0.0)
            value = part / s.double()[:, None]
            got = y[:, at:at + cols].float().double()
            assert ((got - value).abs() <= value.abs() * (2.0 ** -4 + ULP) + 2.0 ** -10).all()
            assert got.abs().amax() <= 448


def test_e4m3_of_zeros_and_next_to_nothing():
    import cfc_recurrent_cell_amd as C
    x = torch.zeros(3, 64, device="cuda")
    x[1] = 1e-37
    w = torch.ones(64, device="cuda")
    y, scales, _ = C.rms_norm_forward_e4m3(x, w, 1.0, group=32)
    assert (scales[0] == torch.tensor(1.0, device="cuda") / 448).all()
    assert (y[0].float() == 0).all() and (y[1].float() == 448).all() and (y[2].float() == 0).all()
    near(scales[1], torch.full((2,), 1e-37 / 448, dtype=torch.float64, device="cuda"), 0.0, floor=2.0 ** -149)


def test_values_that_are_not_finite_stay_in_their_row():
    import cfc_recurrent_cell_amd as C
    for width in (100, 600, 4096):
        x, w, r = make(5, "bf16", 6, width, "same")
        want = C.rms_norm_forward(x, w, EPS, residual=r)
        q = C.rms_norm_forward_e4m3(x, w, EPS, residual=r)
        x[2, 3], x[4, 1] = float("nan"), float("inf")
        got = C.rms_norm_forward(x, w, EPS, residual=r)
        q2 = C.rms_norm_forward_e4m3(x, w, EPS, residual=r)
        keep = [0, 1, 3, 5]
        for a, b in zip((*want, *q), (*got, *q2)):
            assert torch.equal(a[keep].float(), b[keep].float())
        assert torch.isnan(got[0][2]).all() and torch.isnan(got[0][4, 1])
        assert torch.isnan(q2[0][2].float()).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,width", SIZES)
def test_backward(kind, rows, width):
    import cfc_recurrent_cell_amd as C
    for residual, stream in (("same", True), ("fp32", True), ("same", False)):
        say(f"[norm] backward {kind} {rows} {width} {residual} {stream}")
        x, w, r = make(rows + width + 2, kind, rows, width, residual)
        gy, _, gh = make(rows + width + 3, kind, rows, width, residual)
        _, h, rstd = C.rms_norm_forward(x, w, EPS, residual=r)
        gx, gw = C.rms_norm_backward(gy, h, w, rstd, grad_h=gh if stream else None)
        assert gx.dtype == r.dtype and gw.dtype == torch.float32
        n = h.double() * rstd.double()[:, None]
        d = gy.double() * w.double()
        mean = (d * n).mean(-1, keepdim=True)
        want = rstd.double()[:, None] * (d - n * mean)
        size = rstd.double()[:, None] * (d.abs() + n.abs() * (d * n).abs().mean(-1, keepdim=True))
        if stream:
            want = want + gh.double()
            size = size + gh.double().abs()
        near(gx, want, torch.finfo(r.dtype).eps / 2, size=size, floor=floor_of(r.dtype))
        near(gw, (gy.double() * n).sum(0), 0.0, size=(gy.double() * n).abs().sum(0))


def test_backward_matches_differences():
    """Central differences of the forward's formula in float64, in random directions."""
    import cfc_recurrent_cell_amd as C
    for width in (24, 700):
        x, w, r = make(8, "fp32", 5, width, "same")
        gy, _, gh = make(9, "fp32", 5, width, "same")
        _, h, rstd = C.rms_norm_forward(x, w, EPS, residual=r)
        gx, gw = C.rms_norm_backward(gy, h, w, rstd, grad_h=gh)

        def value(hh, ww):
            y = hh / torch.sqrt(hh.square().mean(-1, keepdim=True) + EPS) * ww
            return (y * gy.double()).sum() + (hh * gh.double()).sum()

        for seed in range(3):
            dx, dw, _ = make(20 + seed, "fp32", 5, width, "none")
            dx, dw, step = dx.double(), dw.double(), 1e-5
            num = (value(h.double() + step * dx, w.double() + step * dw) -
                   value(h.double() - step * dx, w.double() - step * dw)) / (2 * step)
            got = (gx.double() * dx).sum() + (gw.double() * dw).sum()
            size = (gx.double() * dx).abs().sum() + (gw.double() * dw).abs().sum()
            assert abs(num - got) <= ULP * size + 1e-8 * size


def test_in_place_and_no_rows():
    import cfc_recurrent_cell_amd as C
    for width in (64, 600, 4096):
        x, w, r = make(10, "bf16", 30, width, "same")
        y, h, rstd = C.rms_norm_forward(x, w, EPS, residual=r)
        r2 = r.clone()
        y2, h2, _ = C.rms_norm_forward(x, w, EPS, residual=r2, h=r2)
        assert h2 is r2 and torch.equal(h2, h) and torch.equal(y2, y)
        gx, gw = C.rms_norm_backward(y, h, w, rstd, grad_h=x)
        x2 = x.clone()
        gx2, gw2 = C.rms_norm_backward(y, h, w, rstd, grad_h=x2, grad_x=x2)
        assert gx2 is x2 and torch.equal(gx2, gx) and torch.equal(gw2, gw)
    none = x[:0]
    y, h, rstd = C.rms_norm_forward(none, w, EPS)
    assert y.shape == none.shape and rstd.shape == (0,)
    gx, gw = C.rms_norm_backward(none, none, w, rstd, grad_weight=torch.full((4096,), 3.0, device="cuda"))
    assert gx.shape == none.shape and (gw == 0).all()


def test_more_leading_axes_and_misaligned_rows():
    import cfc_recurrent_cell_amd as C
    x, w, _ = make(11, "bf16", 24, 80, "none")
    y, _, rstd = C.rms_norm_forward(x, w, EPS)
    y3, _, rstd3 = C.rms_norm_forward(x.view(2, 3, 4, 80), w, EPS)
    assert y3.shape == (2, 3, 4, 80) and torch.equal(y3.view(24, 80), y) and torch.equal(rstd3.view(24), rstd)
    wide = torch.empty(24 * 80 + 1, dtype=x.dtype, device="cuda")
    off = wide[1:].view(24, 80)
    off.copy_(x)
    assert off.data_ptr() % 16 != 0
    y4, _, _ = C.rms_norm_forward(off, w, EPS)
    assert torch.equal(y4, y)


def test_equal_bits_side_stream_and_capture():
    import cfc_recurrent_cell_amd as C
    x, w, r = make(12, "bf16", 700, 1024, "same")
    gy, _, gh = make(13, "bf16", 700, 1024, "same")

    def all_of(**more):
        y, h, rstd = C.rms_norm_forward(x, w, EPS, residual=r, **more)
        q, s, _ = C.rms_norm_forward_e4m3(x, w, EPS, residual=r, group=64, **more)
        return (y, h, rstd, q.view(torch.uint8), s, *C.rms_norm_backward(gy, h, w, rstd, grad_h=gh, **more))

    want = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = all_of(stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_of()
    for seed in range(3):
        x.copy_(make(30 + seed, "bf16", 700, 1024, "none")[0])
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(all_of(), got):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    import cfc_recurrent_cell_amd as C
    rows, width = 140000, 16384
    x, w, _ = make(14, "bf16", 3, width, "none")
    gy, _, gh = make(15, "bf16", 3, width, "same")
    y, h, rstd = C.rms_norm_forward(x, w, EPS)
    gx, gw = C.rms_norm_backward(gy, h, w, rstd)
    many = torch.zeros(rows, width, dtype=x.dtype, device="cuda")
    many[-3:] = x
    y2, _, rstd2 = C.rms_norm_forward(many, w, EPS)
    assert torch.equal(y2[-3:], y) and torch.equal(rstd2[-3:], rstd) and not y2[:-3].any()
    y2.zero_()
    y2[-3:] = gy
    gx2, gw2 = C.rms_norm_backward(y2, many, w, rstd2)
    assert torch.equal(gx2[-3:], gx) and not gx2[:-3].any()
    near(gw2, gw.double(), 0.0, size=(gy.double() * h.double() * rstd.double()[:, None]).abs().sum(0))
    q, s, _ = C.rms_norm_forward_e4m3(many, w, EPS, group=128)
    q3, s3, _ = C.rms_norm_forward_e4m3(x, w, EPS, group=128)
    assert torch.equal(q[-3:].view(torch.uint8), q3.view(torch.uint8)) and torch.equal(s[-3:], s3)
