"""The layer norm's gradients where a row's mean times its rstd passes the range of 32-bit floats,
though what the row's own columns are (differences to the mean) does not: columns behind a
row's end, which its last lanes have, must not get into its sums.

Rows are constant, and sums of so few equal numbers exact, so n = 0, rstd = 1 / sqrt(eps) and
grad_x = rstd * (d - mean(d)): 8 roundings of 2^-24 of rstd * (|d| + mean |d|) at most, and the
output's own."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width", [4, 8, 16, 32])
def test_large_means(gpu, kind, width):
    gen = torch.Generator(device="cuda").manual_seed(width)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(kind)  # noqa: E731
    x, w, b, gy = torch.full((37, width), 2.0 ** 122, device="cuda").to(kind), n(width), n(width), n(37, width)
    y, h, mean, rstd = gpu.layer_norm_forward(x, w, b, EPS)
    assert (mean == 2.0 ** 122).all() and torch.equal(y, b.expand(37, -1))
    gx, gw, gb = gpu.layer_norm_backward(gy, h, w, mean, rstd)
    d, rs = gy.double() * w.double(), EPS ** -0.5
    want = rs * (d - d.mean(-1, keepdim=True))
    room = torch.finfo(kind).eps / 2 * want.abs() + 8 * 2.0 ** -24 * rs * (d.abs() + d.abs().mean(-1, keepdim=True))
    assert ((gx.double() - want).abs() <= room).all()
    assert (gw == 0).all()
    assert ((gb.double() - gy.double().sum(0)).abs() <= 8 * 2.0 ** -24 * gy.double().abs().sum(0)).all()
