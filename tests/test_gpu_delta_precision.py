"""How exactly the delta rule's chunks compute what their types can hold.

Errors are held to what independent roundings give: a value that passes n of them,
each at most 2^-24 of `size` (the largest partial sum) and spread evenly, is off by
sqrt(n / 3) 2^-24 size in the root of the mean square over many outputs."""
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


def rms(t):
    return t.double().square().mean().sqrt().item()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("batch,heads,dk,dv", [(1, 2, 64, 128), (3, 8, 64, 256), (1, 2, 128, 128), (3, 8, 128, 256)])
def test_o_where_a_large_value_is_taken_back(gpu, kind, batch, heads, dk, dv):
    """Every token has the unit key k = q, the gate 1 and no decay, so o = v, however large
    S0^T k is: scale Q S0 and M U cancel.  Roundings on the way to o: dim_k each in S0^T k and
    S0^T q, 64 each in T's and M's products and 32 in the inverse; what products of parts
    leave out is at most 2^-22 of size in the sums before and after U.  Narrow tiles and
    wide ones (384 narrow ones)."""
    say(f"[delta] cancelling o {kind} {batch} {heads} {dk} {dv}")
    gen = torch.Generator().manual_seed(71)
    length, t = 100, TYPES[kind]
    k = torch.zeros(batch, length, heads, dk)
    k[..., ::dk // 64] = 0.125                                      # 64 of them: a unit key in every type
    k = k.to(t).cuda()
    v = (1e-3 * torch.randn(batch, length, heads, dv, generator=gen)).to(t).cuda()
    s0 = (1 + torch.rand(batch, heads, dk, dv, generator=gen)).cuda()
    g = torch.zeros(batch, length, heads, device="cuda")
    o, _ = gpu.delta_rule_forward(k, k, v, g, torch.ones_like(g), initial_state=s0, scale=1.0)
    size = 8 * s0.mean().item()
    step = rms(v) * torch.finfo(t).eps / 2
    bound = ((2 * dk + 160) / 3) ** 0.5 * 2.0 ** -24 * size + 2 * 2.0 ** -22 * size + step
    err = rms(o.double() - v.double())
    assert err <= bound, f"{err:.3e} of {bound:.3e}"


@pytest.mark.parametrize("batch,heads", [(1, 4), (4, 16)])
def test_parts_leave_nothing_out_on_one_side(gpu, batch, heads):
    """o = Q S0 of positive values (a gate of 0 adds nothing), 128 terms a sum, in fp32.  Parts
    that were cut off would leave out 2^-8 2^-16 of each product twice, half of it on average
    and always of one sign: -2^-24.  Rounded parts leave out as much of either sign, and the
    sum's roundings are even, so the mean over more than 2^15 outputs is held to a
    quarter of that; a single value to the roundings of 128 terms."""
    say(f"[delta] parts {batch} {heads}")
    gen = torch.Generator().manual_seed(72)
    length, dim = 64, 128
    q = torch.rand(batch, length, heads, dim, generator=gen) + 0.1
    s0 = torch.rand(batch, heads, dim, dim, generator=gen) + 0.1
    want = (q.double().transpose(1, 2).contiguous() @ s0.double()).transpose(1, 2)
    g = torch.zeros(batch, length, heads, device="cuda")
    o, final = gpu.delta_rule_forward(q.cuda(), q.cuda() / 16, torch.randn(q.shape, generator=gen).cuda(), g, g,
                                      initial_state=s0.cuda(), scale=1.0)
    off = o.double().cpu() / want - 1
    assert abs(off.mean().item()) <= 2.0 ** -26, f"mean {off.mean().item():.3e}"
    assert off.abs().max() <= 128 * 2.0 ** -24
    assert torch.equal(final.cpu(), s0)
