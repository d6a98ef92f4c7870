"""The weight's and the bias's gradients of the short convolution.

Tolerances.  A term is grad_y * y'(p) * x: p's width + 1 terms and its gate are off by 16
roundings of 2^-24 of the terms' magnitudes, the slope by as many, and one more is the product's.
At most 32 terms are added in 32 bits, one after the other (the tokens of a wave), which are 32
roundings, and those sums in 64 bits, rounded once: half a step of the result."""
import pytest

import sequence_reference as R
import test_gpu_short_conv as V
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


# (few tokens and channels, whose waves have 16 tokens, and many, whose have 32)
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("channels,width,lens", [(40, 4, [300, 0, 77]), (513, 3, (2, 200)), (2304, 4, [4100, 30, 4062]), (1030, 2, [17] * 900)])
@pytest.mark.parametrize("activation", ["silu", None])
def test_sums_over_tokens(gpu, kind, channels, width, lens, activation):
    say(f"[conv] sums {kind} {channels} {width} {activation}")
    rows, tokens, count, offsets = V.layout(lens)
    p, on = V.make(channels, kind, tokens, count, channels, width)
    o = {n: t.unflatten(0, lens) if isinstance(lens, tuple) and n in ("x", "gy") else t for n, t in on.items()}
    args = (p["x"], p["w"], p["b"], p["s"], rows, activation is not None, p["gy"], p["gf"])
    want, size = R.conv(*args)[2], R.conv(*args, size=True)[2]
    got = gpu.short_conv_backward(o["x"], o["w"], o["gy"], bias=o["b"], initial_state=o["s"], grad_final_state=o["gf"],
                                  activation=activation, offsets=offsets)
    V.near("weight", got[1], want["weight"], size["weight"], 65)
    V.near("bias", got[2], want["bias"], size["bias"], 65)
