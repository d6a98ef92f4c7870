"""The selective scan over rows that lie far apart, as those of one batch row of a time-major
tensor do: the longest strides that are accepted, on both sides of where the forward of few
workgroups changes its kernel, over several blocks of tokens and with states that do not fill
a lane's.  Reference and tolerances are those of test_gpu_selective_scan.py."""
import pytest

import sequence_reference as R
import test_gpu_selective_scan as S
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


# bytes that this many rows span: just under what is accepted, and under what 128 rows of a block reach
@pytest.mark.parametrize("rows", [64, 128])
@pytest.mark.parametrize("kind,channels,groups,state", [("bf16", 40, 1, 5), ("fp32", 24, 2, 3), ("fp16", 16, 1, 8), ("bf16", 20, 1, 16)])
def test_longest_strides(gpu, rows, kind, channels, groups, state):
    say(f"[scan] strides {rows} {kind} {channels} {groups} {state}")
    tokens, t = 270, S.TYPES[kind]
    stride = (1 << 31) // (rows * t.itemsize) - channels - state - 1
    gen, p, on = S.inputs(state, kind, tokens, 1, channels, groups, state)
    gy, on["gy"] = S.some(gen, t, (tokens, channels))
    far = torch.empty(tokens, stride, device="cuda", dtype=t)  # 9 GB at most; the columns read are written below
    at, views = 0, {}
    for n in ("x", "dt", "z", "gy", "b", "c"):
        flat = on[n].flatten(1)
        views[n] = far[:, at:at + flat.shape[1]]
        views[n].copy_(flat)
        if n in "bc":
            views[n] = views[n].unflatten(-1, (groups, state))
        at += flat.shape[1] + 3
    far[:, at:at + 64] = float("nan")  # behind the last rows' columns
    one = {n: v[None] for n, v in views.items()}
    args, more = (one["x"], one["dt"], on["a"], one["b"], one["c"]), dict(d=on["d"], z=one["z"], dt_bias=on["dt_bias"])
    y, final = gpu.selective_scan_forward(*args, initial_state=on["initial"], **more)
    rows_of, ulps = R.spans([tokens]), S.roundings(p, R.spans([tokens]), True)
    gf = R.np.zeros_like(p["initial"])
    want, wf, wg = R.scan(p, rows_of, True, gy, gf)
    size, sf, sg = R.scan(p, rows_of, True, gy, gf, size=True)
    S.near(("y", y.dtype), y, want, size, ulps)
    S.near(("final", final.dtype), final, wf, sf, ulps)
    got = gpu.selective_scan_backward(*args, one["gy"], initial_state=on["initial"], **more)
    for n, g in zip(R.NAMES, got):
        S.near((n, g.dtype), g, wg[n], sg[n], ulps)
    # the dense rows' gradients are the same kernels', and so are the outputs where their blocks are
    dense = {n: v.contiguous() for n, v in one.items()}
    args, more = (dense["x"], dense["dt"], on["a"], dense["b"], dense["c"]), {**more, "z": dense["z"]}
    for u, v in zip(got, gpu.selective_scan_backward(*args, dense["gy"], initial_state=on["initial"], **more)):
        assert torch.equal(u, v)
    if rows == 128 or state > 8:
        for u, v in zip((y, final), gpu.selective_scan_forward(*args, initial_state=on["initial"], **more)):
            assert torch.equal(u, v)
