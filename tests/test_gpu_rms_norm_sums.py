"""The norm's weight gradient over so many rows that a workgroup's own sum is long."""
import pytest

from parity_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


@pytest.mark.parametrize("rows,width,kind", [(1 << 22, 128, torch.bfloat16), (1 << 20, 512, torch.float32),
                                             (400001, 1024, torch.float16), (1 << 19, 2048, torch.bfloat16),
                                             (100003, 4096, torch.bfloat16)])
def test_weight_gradient_of_many_rows(gpu, rows, width, kind):
    """All rows alike, so that no rounding is made up for by another: 200 to 512 rows a slot.  Four
    roundings of 2^-24 are allowed, of h * rstd, of its product, of a workgroup's sum and of
    the result."""
    say(f"[norm] weight gradient {rows} {width} {kind}")
    gen = torch.Generator(device="cuda").manual_seed(91)
    h1 = torch.rand(width, generator=gen, device="cuda").add(0.1).to(kind)
    gy1 = torch.rand(width, generator=gen, device="cuda").add(0.1).to(kind)
    weight = torch.ones(width, device="cuda", dtype=kind)
    h, gy = h1.expand(rows, width).contiguous(), gy1.expand(rows, width).contiguous()
    rstd = torch.full((rows,), 1.2345678, device="cuda")
    _, gw = gpu.rms_norm_backward(gy, h, weight, rstd)
    want = rows * (gy1.double() * h1.double() * rstd[0].double())
    off = ((gw.double() - want) / want).abs().max().item()
    assert off <= 4 * 2.0 ** -24, f"{off:.3e}"
