"""Clipping where the norm passes the range of 32-bit floats, though its 64-bit root does not:
the caller gets an infinite norm, so the factor is 0; with an infinite max_norm it is 1."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
LISTS = {"one": [(9, torch.float32)], "mixed": [(1, torch.float32), (4, torch.bfloat16), (100, torch.float16)],
         "batches": [(1, torch.float32)] * 120 + [(3, torch.bfloat16)] * 120}  # more than a launch takes


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


@pytest.mark.parametrize("name", LISTS)
def test_a_norm_past_32_bits(gpu, name):
    grads = [torch.full((n,), 60000.0 if t == torch.float16 else 3e38, dtype=t, device="cuda") for n, t in LISTS[name]]
    exact = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert torch.finfo(torch.float32).max < exact < math.inf
    for top in (1e38, 1.0, 0.0):
        out = [torch.full_like(g, 5.0) for g in grads]
        assert math.isinf(float(gpu.clip_grad_norm(grads, top, out=out)))
        assert all((o == 0).all() for o in out), top
    out = [torch.full_like(g, 5.0) for g in grads]
    assert math.isinf(float(gpu.clip_grad_norm(grads, math.inf, out=out)))
    assert all(torch.equal(o, g) for o, g in zip(out, grads))


def test_infinite_gradients_with_an_infinite_limit(gpu):
    grads = [torch.tensor([1.0, math.inf, -2.0], device="cuda"), torch.tensor([3.0], device="cuda")]
    out = [torch.empty_like(g) for g in grads]
    assert math.isinf(float(gpu.clip_grad_norm(grads, math.inf, out=out)))
    assert all(torch.equal(o, g) for o, g in zip(out, grads))


def test_the_largest_norm_within_32_bits_clips(gpu):
    top = torch.finfo(torch.float32).max
    g = torch.tensor([top], device="cuda")
    norm = gpu.clip_grad_norm([g], 1e38)
    assert float(norm) == top
    # the factor is rounded to 32 bits, and the product: 2^-24 each
    assert abs(float(g) - 1e38) <= 2.0 ** -22 * 1e38
