"""Rows behind the last packed sequence (a batch padded to a fixed number of tokens)."""
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


@pytest.mark.parametrize("lens,pad", [([70, 3], 55), ([3, 2], 20), ([0, 0], 64)])
def test_rows_behind_the_last_sequence_are_zeros_in_a_new_buffer(gpu, lens, pad):
    """The memory that a new buffer gets held NaN; a norm over all rows, and its weight
    gradient, stay finite."""
    say(f"[delta] padded {lens} {pad}")
    gen = torch.Generator(device="cuda").manual_seed(61)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    used, rows = sum(lens), sum(lens) + pad
    q, k = (torch.nn.functional.normalize(n(rows, 2, 64), dim=-1).bfloat16() for _ in range(2))
    v, go = n(rows, 4, 64).bfloat16(), n(rows, 4, 64).bfloat16()
    g, beta = -n(rows, 4).abs(), torch.sigmoid(n(rows, 4))
    offsets = torch.tensor([0, lens[0], used], dtype=torch.int32, device="cuda")
    weight = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    for _ in range(2):
        stale = [torch.full_like(t, float("nan")) for t in (v, v, q, q, g, g)]
        torch.cuda.synchronize()
        del stale
        o, _ = gpu.delta_rule_forward(q, k, v, g, beta, offsets=offsets)
        assert (o[used:] == 0).all() and torch.isfinite(o).all()
        for t in gpu.delta_rule_backward(q, k, v, g, beta, go, offsets=offsets)[:5]:
            assert (t[used:] == 0).all() and torch.isfinite(t).all()
        _, _, rstd = gpu.rms_norm_forward(o, weight, 1e-6)
        _, grad = gpu.rms_norm_backward(go, o, weight, rstd)
        assert torch.isfinite(grad).all()
