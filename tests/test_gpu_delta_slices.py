"""The delta rule over a few tokens of a long tensor: rows so far apart that 64 of them
pass 2^31 bytes give the bits that contiguous ones give."""
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


def rows(batch, length, far):
    """q, k, v, grad_o, g, beta; the first four with the tokens `far` elements apart."""
    gen = torch.Generator(device="cuda").manual_seed(81)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    wide = torch.empty(batch * length, far, dtype=torch.bfloat16, device="cuda")
    out, at = [], 0
    for heads in (2, 2, 4, 4):
        t = wide[:, at:at + heads * 64].view(batch, length, heads, 64)
        t.copy_(torch.nn.functional.normalize(n(batch, length, heads, 64), dim=-1))
        at += heads * 64
        out.append(t)
    return (*out, -n(batch, length, 4).abs(), torch.sigmoid(n(batch, length, 4)))


@pytest.mark.parametrize("batch,length", [(1, 1), (3, 1), (1, 5), (2, 3)])
def test_few_rows_far_apart(gpu, batch, length):
    say(f"[delta] {batch} x {length} rows far apart")
    q, k, v, go, g, beta = rows(batch, length, (1 << 24) + 64)
    assert batch * length == 1 or q.stride(1 if length > 1 else 0) > 1 << 24
    close = [t.contiguous() for t in (q, k, v)]
    got = gpu.delta_rule_forward(q, k, v, g, beta)
    for x, y in zip(got, gpu.delta_rule_forward(*close, g, beta)):
        assert torch.equal(x, y)
    if length > 1:
        with pytest.raises(ValueError, match="2\\^31 bytes"):
            gpu.delta_rule_backward(q, k, v, g, beta, go)
        return
    got = gpu.delta_rule_backward(q, k, v, g, beta, go)
    for x, y in zip(got[:5], gpu.delta_rule_backward(*close, g, beta, go.contiguous())):
        assert torch.equal(x, y)


def test_one_token_of_a_long_tensor(gpu):
    """x[:, t:t + 1] of one sequence: the batch's stride is that of all 8192 tokens."""
    gen = torch.Generator(device="cuda").manual_seed(82)
    x = torch.nn.functional.normalize(torch.randn(1, 8192, 16, 128, generator=gen, device="cuda"), dim=-1).bfloat16()
    t = x[:, 77:78]
    g = torch.full((1, 1, 16), -0.1, device="cuda")
    got = (*gpu.delta_rule_forward(t, t, t, g, -g), *gpu.delta_rule_backward(t, t, t, g, -g, t)[:5])
    c = t.clone(memory_format=torch.contiguous_format)
    for a, b in zip(got, (*gpu.delta_rule_forward(c, c, c, g, -g), *gpu.delta_rule_backward(c, c, c, g, -g, c)[:5])):
        assert torch.equal(a, b)


def test_sizes_that_are_refused(gpu):
    """Empty heads, and a pool of more states than 32 bits count (its low 32 bits would be five)."""
    for dk, dv, heads in ((0, 8, 2), (8, 0, 2), (8, 8, 0)):
        q, v = (torch.zeros(1, 3, h, d, device="cuda") for h, d in ((2, dk), (heads, dv)))
        g = torch.zeros(1, 3, heads, device="cuda")
        with pytest.raises(ValueError, match="elements|heads"):
            gpu.delta_rule_forward(q, q, v, g, g)
        with pytest.raises(ValueError, match="elements|heads"):
            gpu.delta_rule_step(q[0], q[0], v[0], g[0], g[0], torch.zeros(3, heads, dk, dv, device="cuda"))
    q, g = torch.zeros(5, 1, 1, device="cuda"), torch.zeros(5, 1, device="cuda")
    many = torch.empty((1 << 32) + 5, 1, 1, 1, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        gpu.delta_rule_step(q, q, q, g, g, many)
