"""The delta rule's kernels for large calls, which a rule on the sizes chooses: wide
tiles of dim_v (more than 256 narrow ones, 384 where the gradients' chains share a
launch, 768 for a forward in bf16), packed batches of more sequences than a wave has lanes, steps whose states
pass the cache by, sequences of many chunks; and keys that are not unit vectors.

Tolerances are those of test_gpu_delta_rule.py, without its allowance for 16-bit o.  Along
a sequence a chunk's error is kept with its state: decays here are at least 0.025 a token on
average, so a chunk keeps a fifth of the one before and all of them together 1.25 times
one chunk's bound, of which the bound's worst case (every rounding of one sign) has
room for many."""
import numpy as np
import pytest

from parity_util import say
from test_gpu_delta_rule import Case, step_case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


def check(c):
    """Forward and gradients of a Case; a gate's gradient is a difference of sums, of u and of S k."""
    want_o, want_s = c.want_forward()
    o, final = c.forward()
    c.near(o, want_o, "o")
    c.near(final, want_s, "final")
    want, mag = c.want_backward()
    for n, t in zip(("q", "k", "v", "g", "beta", "initial"), c.backward()):
        if t is not None:
            size = max(mag.max(), np.abs(want[n]).max()) if n in ("g", "beta") else None
            c.near(t, want[n], n, size=size)


LENS = [66, 1, 0, 64, 65, 33, 7, 70, 130, 2, 64, 9, 63]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("hk,hv,dk,dv", [(2, 4, 128, 128), (4, 4, 64, 128), (2, 4, 100, 130), (1, 4, 33, 117),
                                         (4, 8, 128, 128), (8, 8, 64, 128), (2, 8, 100, 130), (1, 8, 33, 117)])
def test_wide_tiles(kind, hk, hv, dk, dv):
    assert len(LENS) * hv * -(-dv // 16) > (768 if hv == 8 else 384)
    say(f"[delta] wide {kind} {hk} {hv} {dk} {dv}")
    check(Case(101, kind, lens=LENS, hk=hk, hv=hv, dk=dk, dv=dv))


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_wide_tiles_of_equal_sequences(kind):
    say(f"[delta] wide dense {kind}")
    check(Case(102, kind, batch=49, length=70, hk=1, hv=2, dk=64, dv=128, state=False))
    check(Case(103, kind, batch=25, length=65, hk=1, hv=2, dk=128, dv=256))


@pytest.mark.parametrize("count", [64, 65, 200, 5000])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_many_packed_sequences(count, kind):
    """Mostly empty ones and single tokens, a few of some chunks, the last one among them."""
    say(f"[delta] {count} packed sequences {kind}")
    lens = np.random.default_rng(count).choice([0, 0, 1, 1, 2, 3], count).tolist()
    lens[0], lens[count // 3], lens[-1] = 0, 150, 129
    check(Case(104, kind, lens=lens, hk=1, hv=2, dk=16, dv=24))


@pytest.mark.parametrize("kind,length,hk,hv,dk,dv", [("bf16", 4100, 1, 1, 128, 128), ("fp16", 3001, 1, 2, 64, 40),
                                                     ("fp32", 3001, 1, 1, 128, 64), ("bf16", 2049, 2, 2, 64, 16)])
def test_many_chunks(kind, length, hk, hv, dk, dv):
    say(f"[delta] {length} tokens {kind} {hk} {hv} {dk} {dv}")
    check(Case(105, kind, batch=1, length=length, hk=hk, hv=hv, dk=dk, dv=dv))


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dk", [16, 64, 128])
def test_keys_of_any_length(kind, dk):
    """Keys and queries of normal numbers, |k|^2 about dim_k; gates below 1 / dim_k keep the rule stable."""
    say(f"[delta] keys of any length {kind} {dk}")
    check(Case(106, kind, lens=[100, 3, 64, 200], hk=2, hv=4, dk=dk, dv=48, k_norm=False, beta_top=1 / dk))


@pytest.mark.parametrize("kind,batch,hk,hv,dk,dv", [("bf16", 256, 8, 16, 128, 128), ("fp16", 200, 16, 32, 128, 67),
                                                    ("fp32", 256, 64, 64, 33, 100), ("bf16", 1600, 8, 64, 16, 32)])
def test_steps_past_the_cache(gpu, kind, batch, hk, hv, dk, dv):
    """192 MB of states and more, some rows idle and some of one slot, against the same rows 25 at a time."""
    assert batch * hv * dk * dv * 4 >= 192 << 20 > 25 * hv * dk * dv * 4
    say(f"[delta] step past the cache {kind} {batch} {hk} {hv} {dk} {dv}")
    r = np.random.default_rng(107)
    slots = r.permutation(batch + 10)[:batch]
    slots[3], slots[batch // 2], slots[-1], slots[7] = -1, slots[5], slots[5], batch + 10
    c, args, _, sl = step_case(107, kind, batch, 1, hk, hv, dk, dv, slots.tolist())
    gen = torch.Generator(device="cuda").manual_seed(107)
    states = torch.randn(batch + 10, hv, dk, dv, generator=gen, device="cuda")
    few = states.clone()
    o = gpu.delta_rule_step(*args, states, slots=sl)
    for at in range(0, batch, 25):
        part = [t[at:at + 25].contiguous() for t in args]
        assert torch.equal(o[at:at + 25], gpu.delta_rule_step(*part, few, slots=sl[at:at + 25].contiguous()))
    assert torch.equal(states, few)
    # and in order, without slots
    o = gpu.delta_rule_step(*args, states)
    for at in range(0, batch, 25):
        part = [t[at:at + 25].contiguous() for t in args]
        assert torch.equal(o[at:at + 25], gpu.delta_rule_step(*part, few[at:at + 25]))
    assert torch.equal(states, few)
