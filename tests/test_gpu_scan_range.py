"""The selective scan where its stretches' products leave the range of 32-bit floats, though the
recurrence token by token does not: steps whose sum over a stretch is infinite beside rates of
exactly zero and states that do not fill a lane's, and decays whose product is infinite where
the state, or its gradient, is zero.

Tolerances.  Steps are taken as they are (no softplus), so nothing grows with their size:
decays are 0, 1 or of exponents below one.  A token adds 4 roundings of 2^-24 to a state and 4 to
its gradient, 64 are for the rest, as in test_gpu_selective_scan.py."""
import numpy as np
import pytest

import sequence_reference as R
import test_gpu_selective_scan as S
from parity_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TOKENS = 77
# the states of a lane, few workgroups (a sequence) and many
CASES = [(kind, state, count) for kind in ("fp32", "bf16") for state in (3, 4, 5, 12, 16, 30, 50) for count in (1, 300) if count == 1 or state in (5, 12)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


def make(state, count):
    channels = 16
    gen = np.random.default_rng(state)
    n = gen.standard_normal
    p = {"x": n((count, TOKENS, channels)), "dt": 0.01 + 0.01 * np.abs(n((count, TOKENS, channels))), "a": -np.exp(n((channels, state))),
         "b": n((count, TOKENS, 1, state)), "c": n((count, TOKENS, 1, state)), "gy": n((count, TOKENS, channels)), "d": None, "z": None,
         "dt_bias": None, "initial": np.zeros((count, channels, state)), "gf": np.zeros((count, channels, state))}
    return p


def run(gpu, kind, p):
    """Forward and gradients, both held to the reference; the gradients."""
    rows = R.spans(batch=len(p["x"]), length=TOKENS)
    on, q = {}, {}
    for n, v in p.items():
        if v is None:
            on[n] = q[n] = None
            continue
        t = torch.from_numpy(v).to(S.TYPES[kind] if n in (*S.ROWS, "gy") else torch.float32)
        on[n], q[n] = t.cuda(), t.double().numpy()
        if n in (*S.ROWS, "gy"):
            q[n] = q[n].reshape(-1, *v.shape[2:])
    args = [on[n] for n in ("x", "dt", "a", "b", "c")]
    y, final = gpu.selective_scan_forward(*args, initial_state=on["initial"], softplus=False)
    got = gpu.selective_scan_backward(*args, on["gy"], initial_state=on["initial"], grad_final_state=on["gf"], softplus=False)
    with np.errstate(under="ignore"):
        want, wf, wg = R.scan(q, rows, False, q["gy"], q["gf"])
        size, sf, sg = R.scan(q, rows, False, q["gy"], q["gf"], size=True)
    assert all(np.isfinite(v).all() for v in (want, wf, *wg.values()))
    ulps = (64 + 8 * TOKENS) * 2.0 ** -24
    S.near(("y", y.dtype), y, want, size, ulps)
    S.near(("final", final.dtype), final, wf, sf, ulps)
    for n, g in zip(R.NAMES, got):
        if g is not None:
            S.near((n, g.dtype), g, wg[n], sg[n], ulps)
    return y, got


@pytest.mark.parametrize("kind,state,count", CASES)
def test_steps_whose_sum_is_infinite(gpu, kind, state, count):
    """They forget every state but those of a rate of zero, which gather what is added."""
    say(f"[scan] range of steps {kind} {state} {count}")
    p = make(state, count)
    p["a"][:, 0] = 0.0
    long = slice(10, 40)
    p["dt"][:, long] = 3e38
    p["x"][:, long] *= 1e-38
    p["gy"] *= 1e-20  # the gradients of such steps' rates are products with them
    y, _ = run(gpu, kind, p)
    assert float(y[:, 41:].float().abs().max()) > 0.1


@pytest.mark.parametrize("kind,state,count", CASES)
def test_products_of_decays_that_are_infinite(gpu, kind, state, count):
    """States grow by exp(30) a token, and are zero meanwhile."""
    say(f"[scan] range of decays {kind} {state} {count}")
    p = make(state, count)
    p["a"] = np.full_like(p["a"], 30.0)
    p["dt"][:, :37], p["x"][:, :37] = 1.0, 0.0
    p["gy"][:] = 0
    y, _ = run(gpu, kind, p)
    assert (y[:, :37] == 0).all() and float(y[:, 38:].float().abs().max()) > 0.01
    # and their gradients are zero: from the tokens that grow on, nothing is asked for
    p = make(state, count)
    p["a"] = np.full_like(p["a"], 30.0)
    p["x"][:] = 0
    p["dt"][:, 40:], p["gy"][:, 40:] = 1.0, 0.0
    _, got = run(gpu, kind, p)
    assert (got[0][:, 40:] == 0).all() and float(got[0][:, :39].float().abs().max()) > 0.01
