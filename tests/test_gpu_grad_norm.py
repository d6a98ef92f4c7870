"""The norm over many gradients and clipping on the GPU against their formula in float64.

Tolerances.  The sum of squares is taken in 64 bits, so the norm is its root rounded to 32:
2^-24 of it, and a little (2^-40) for the sums.  A clipped gradient is g times the factor,
rounded to 32 bits, which is one more rounding, and then rounded to its type."""
import math

import pytest

from parity_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


def make(seed, sizes, kinds, scale=1e-2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(scale * torch.randn(n, generator=g, device="cuda")).to(TYPES[kinds[i % len(kinds)]]) for i, n in enumerate(sizes)]


def norm_of(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def held(got, grads, norm, max_norm):
    factor = min(1.0, max_norm / (norm + 1e-6))
    for i, (o, g) in enumerate(zip(got, grads)):
        want = g.double() * factor
        tiny = 2.0 ** -25 if g.dtype == torch.float16 else 2.0 ** -149
        room = (torch.finfo(g.dtype).eps / 2 + 2 * 2.0 ** -24) * want.abs() + tiny
        assert o.dtype == g.dtype and o.shape == g.shape
        assert ((o.double() - want).abs() <= room).all(), i


LISTS = [([1], ["fp32"]), ([0, 5, 0], ["bf16"]), ([16384, 16384, 128, 128], ["fp32"]), ([7, 8, 9, 2047, 2048, 2049], ["bf16", "fp32", "fp16"]),
         ([3] * 300, ["fp32", "bf16"]), ([0] * 113 + [5000], ["fp16"]), ([9_000_001, 3], ["bf16"]), ([100_003] * 230, ["bf16", "fp32"])]


@pytest.mark.parametrize("sizes,kinds", LISTS, ids=[f"{len(s)}_of_{max(s)}" for s, _ in LISTS])
def test_norm_and_clip(gpu, sizes, kinds):
    say(f"[clip] {len(sizes)} of {max(sizes)} {kinds}")
    grads = make(len(sizes), sizes, kinds)
    want = norm_of(grads)
    norm = gpu.grad_norm(grads)
    assert norm.shape == () and norm.dtype == torch.float32
    assert abs(float(norm) - want) <= (2.0 ** -24 + 2.0 ** -40) * want
    for max_norm in (0.5 * want, 2 * want + 1, 0.0, float("inf")):
        kept = [g.clone() for g in grads]
        out = [torch.full_like(g, 3.0) for g in grads]
        got = gpu.clip_grad_norm(grads, max_norm, out=out)
        assert torch.equal(got, norm)
        assert all(torch.equal(g, k) for g, k in zip(grads, kept))
        held(out, grads, want, max_norm)
        own = [g.clone() for g in grads]
        assert torch.equal(gpu.clip_grad_norm(own, max_norm), norm)
        assert all(torch.equal(o, u) for o, u in zip(own, out))


def test_shapes_addresses_and_names(gpu):
    base = torch.randn(5000, device="cuda").bfloat16()
    grads = [base[1:1001].view(10, 100), base[1002:1003].view(()), base[1005:4000]]
    flat = [g.clone() for g in grads]
    want = norm_of(grads)
    around = base.clone()
    norm = torch.zeros((), device="cuda")
    assert gpu.clip_grad_norm(grads, 1.0, norm=norm) is norm
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    held(grads, flat, want, 1.0)
    for i in (0, 1001, 1003, 1004, *range(4000, 5000)):
        assert base[i] == around[i]
    twice = gpu.grad_norm([flat[0], flat[0]])
    assert abs(float(twice) - math.sqrt(2) * norm_of(flat[:1])) <= 2.0 ** -22 * float(twice)
    assert float(gpu.grad_norm([], norm=norm)) == 0.0
    assert float(gpu.clip_grad_norm([], 1.0, norm=norm)) == 0.0
    assert float(gpu.clip_grad_norm([flat[0][:0]], 1.0)) == 0.0


def test_large_small_and_not_finite(gpu):
    big = [torch.full((3000,), 1e30, device="cuda"), torch.full((5,), 3e38, device="cuda").bfloat16()]
    want = norm_of(big)
    # sqrt(5) * 3.004e38 = 6.7e38 passes 32 bits' 3.4e38; the first tensor and one of the five do not
    assert want > torch.finfo(torch.float32).max and math.isinf(float(gpu.grad_norm(big)))
    big[1] = big[1][:1]
    want = norm_of(big)
    assert abs(float(gpu.grad_norm(big)) - want) <= 2.0 ** -23 * want
    assert math.isinf(float(gpu.grad_norm([torch.full((9,), 3e38, device="cuda")])))
    small = [torch.full((3000,), 1e-30, device="cuda")]
    assert abs(float(gpu.grad_norm(small)) - norm_of(small)) <= 2.0 ** -23 * norm_of(small)
    g = make(3, [100, 5000], ["fp32"])
    g[1][77] = float("inf")
    out = [torch.empty_like(t) for t in g]
    assert math.isinf(float(gpu.clip_grad_norm(g, 1.0, out=out)))
    assert (out[0] == 0).all() and torch.isnan(out[1][77]) and (out[1][:77] == 0).all()
    g[0][3] = float("nan")
    for top in (1.0, float("inf")):
        assert math.isnan(float(gpu.clip_grad_norm(g, top, out=out)))
        assert all(torch.isnan(o).all() for o in out)


def test_the_cells_gradients_are_clipped(gpu):
    """A training step of the CfC cell: backward, reduce_axis0, and the clipping of its sum."""
    from cfc_recurrent_cell_amd import workloads as W
    inp = W.make_cfc_inputs(W.TINY)
    on = [torch.from_numpy(getattr(inp, n)).cuda() for n in ("w_in", "w_rec", "b", "w_tau", "x", "h0", "y")]
    _, scratch, _ = gpu.cfc_forward_backward(*on, float(inp.dt))
    total = gpu.reduce_axis0(scratch)
    sizes = [t.numel() for t in on[:4]]
    parts = list(total.split(sizes))
    kept = [p.clone() for p in parts]
    want = norm_of(kept)
    norm = gpu.clip_grad_norm(parts, 0.1 * want)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    held(parts, kept, want, 0.1 * want)
    assert abs(float(total.double().norm()) - 0.1 * want) <= 1e-5 * want


def test_equal_bits_on_another_stream_and_replayed(gpu):
    grads = make(5, [70000, 3, 128, 200001], ["fp32", "bf16"])

    def work():
        out = [torch.empty_like(g) for g in grads]
        return [gpu.grad_norm(grads), gpu.clip_grad_norm(grads, 0.7, out=out), *out]

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
        kept = work()
    start = [g.clone() for g in grads]
    for i in range(3):
        for g, s in zip(grads, start):
            g.copy_(s * (i + 1))
        eager = [t.clone() for t in work()]
        for t in kept:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(eager, kept))
