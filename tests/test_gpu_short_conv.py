"""The short causal convolution on the GPU against its formula in float64.

Tolerances.  An output is rounded once to its type (half a step of the value); before, p is
a sum of width + 1 terms in 32 bits and its gate takes an exponential, a reciprocal and two
products: 16 roundings of 2^-24 of the terms' magnitudes times |y'(p)| (which is up to
1 + |p| times y / p), and as many for the slope, times |y''(p)|.  A
gradient of x adds width + 1 of those.  The weights' gradients are sums over 64 tokens in 32
bits, one after the other, and of those in 64: 64 more."""
import numpy as np
import pytest

import sequence_reference as R
from parity_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ULP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


def near(name, got, want, size, ulps):
    half = torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -149
    got = got.double().cpu().numpy().reshape(want.shape)
    bad = ~(np.abs(got - want) <= half * np.abs(want) + ulps * ULP * size + tiny)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.abs(got - want).max():.3e}"


def make(seed, kind, tokens, count, channels, width):
    gen = np.random.default_rng(seed)
    out, on = {}, {}
    for n, shape in (("x", (tokens, channels)), ("w", (channels, width)), ("b", (channels,)), ("s", (count, width - 1, channels)),
                     ("gy", (tokens, channels)), ("gf", (count, width - 1, channels))):
        t = torch.from_numpy(gen.standard_normal(shape)).to(TYPES[kind])
        out[n], on[n] = t.double().numpy(), t.cuda()
    return out, on


def layout(lens):
    if isinstance(lens, tuple):
        return R.spans(batch=lens[0], length=lens[1]), lens[0] * lens[1], lens[0], None
    ends = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    return R.spans(lens), sum(lens), len(lens), ends


SIZES = [  # channels, width, lengths (packed) or (batch, length)
    (1, 4, [1]), (8, 4, (2, 16)), (512, 4, [64]), (513, 3, [63, 2]), (100, 2, [1, 1, 1, 0, 40]), (7, 3, (3, 1)),
    (1030, 4, [0, 3, 2, 1, 0, 130, 5]), (24, 4, (2, 200)), (600, 2, (1, 65)), (40, 4, [1] * 150 + [0] * 70 + [3]), (16, 4, [0, 0, 15, 17, 64]),
]


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("channels,width,lens", SIZES)
def test_forward_and_backward(gpu, kind, channels, width, lens):
    rows, tokens, count, offsets = layout(lens)
    for act, full in (("silu", True), (None, True), ("silu", False)):
        say(f"[conv] {kind} {channels} {width} {lens} {act} {full}")
        p, on = make(channels + width, kind, tokens, count, channels, width)
        if not full:
            p["b"], p["s"], p["gf"] = None, 0 * p["s"], 0 * p["gf"]
        o = {n: t.unflatten(0, lens) if isinstance(lens, tuple) and n in ("x", "gy") else t for n, t in on.items()}
        opt = {n: o[m] if full else None for n, m in (("bias", "b"), ("initial_state", "s"))}
        y, final = gpu.short_conv_forward(o["x"], o["w"], activation=act, offsets=offsets, **opt)
        args = (p["x"], p["w"], p["b"], p["s"], rows, act is not None, p["gy"], p["gf"])
        want, wf, wg = R.conv(*args)
        size, _, sg = R.conv(*args, size=True)
        assert y.dtype == final.dtype == TYPES[kind]
        near("y", y, want, size, 16)
        np.testing.assert_array_equal(final.double().cpu().numpy(), wf)
        got = gpu.short_conv_backward(o["x"], o["w"], o["gy"], activation=act, offsets=offsets,
                                      grad_final_state=o["gf"] if full else None, **opt)
        assert got[1].dtype == torch.float32
        for n, t, more in zip(("x", "weight", "bias", "initial"), got, (width + 33, 97, 97, width + 33)):
            if not full and n in ("bias", "initial"):
                assert t is None
            else:
                near(n, t, wg[n], sg[n], more)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("channels,width,batch,pool", [(1, 4, 1, 1), (513, 4, 5, 9), (40, 3, 140, 64), (1024, 2, 3, 3)])
def test_step(gpu, kind, channels, width, batch, pool):
    say(f"[conv] step {kind} {channels} {width} {batch} {pool}")
    p, on = make(batch, kind, batch, pool, channels, width)
    gen = np.random.default_rng(2)
    slots = gen.permutation(np.resize(np.arange(pool), max(batch, pool)))[:batch]
    if batch > 2:
        slots[1], slots[-1] = -1, pool
    for act, bias in (("silu", True), (None, False)):
        states, want, size = p["s"].copy(), np.zeros((batch, channels)), np.zeros((batch, channels))
        for i, s in enumerate(slots):
            if 0 <= s < pool:
                a = (p["x"][i:i + 1], p["w"], p["b"] if bias else None, states[s:s + 1], R.spans([1]), act is not None)
                size[i] = R.conv(*a, size=True)[0]
                want[i], states[s] = (v[0] for v in R.conv(*a)[:2])
        held = on["s"].clone()
        y = gpu.short_conv_step(on["x"], on["w"], held, slots=torch.tensor(slots, dtype=torch.int32).cuda(),
                                bias=on["b"] if bias else None, activation=act)
        near("y", y, want, size, 16)
        np.testing.assert_array_equal(held.double().cpu().numpy(), states)
    if batch <= pool:
        held = on["s"].clone()
        y = gpu.short_conv_step(on["x"], on["w"], held, bias=on["b"])
        one = gpu.short_conv_forward(on["x"][:, None], on["w"], bias=on["b"], initial_state=on["s"][:batch])
        assert torch.equal(y, one[0][:, 0]) and torch.equal(held[:batch], one[1])


def test_slices_and_given_buffers(gpu):
    lens = [40, 0, 33, 2]
    _, used, count, offsets = layout(lens)
    p, on = make(5, "bf16", 90, count, 60, 4)
    wide = torch.full((90, 70), 9.0, device="cuda", dtype=torch.bfloat16)
    wide[:, 5:65] = on["x"]
    y, final = gpu.short_conv_forward(on["x"], on["w"], bias=on["b"], initial_state=on["s"], offsets=offsets)
    assert (y[used:] == 0).all()
    given, state = torch.full_like(y, 5.0), on["s"].clone()
    y2, f2 = gpu.short_conv_forward(wide[:, 5:65], on["w"], bias=on["b"], initial_state=state, offsets=offsets, y=given,
                                    final_state=state)
    assert y2 is given and f2 is state and torch.equal(y2[:used], y[:used]) and torch.equal(state, final)
    assert (y2[used:] == 5).all()
    args = dict(bias=on["b"], initial_state=on["s"], grad_final_state=on["gf"], offsets=offsets)
    want = gpu.short_conv_backward(on["x"], on["w"], on["gy"], **args)
    assert (want[0][used:] == 0).all()
    given = torch.full_like(y, 5.0)
    twice = torch.cat([on["gy"], on["gy"]], 1)
    got = gpu.short_conv_backward(wide[:, 5:65], on["w"], twice[:, 60:], grad_x=given, **args)
    assert torch.equal(given[:used], want[0][:used]) and (given[used:] == 5).all()
    assert all(torch.equal(u, v) for u, v in zip(want[1:], got[1:]))


def test_nothing_to_do(gpu):
    p, on = make(6, "fp32", 0, 2, 12, 4)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    y, final = gpu.short_conv_forward(on["x"], on["w"], initial_state=on["s"], offsets=none)
    assert y.shape == (0, 12) and torch.equal(final, on["s"])
    g = gpu.short_conv_backward(on["x"], on["w"], on["gy"], bias=on["b"], initial_state=on["s"], grad_final_state=on["gf"], offsets=none)
    assert (g[1] == 0).all() and (g[2] == 0).all() and torch.equal(g[3], on["gf"])
    p, on = make(6, "fp32", 5, 0, 12, 4)
    y, _ = gpu.short_conv_forward(on["x"], on["w"], offsets=none[:1])
    g = gpu.short_conv_backward(on["x"], on["w"], on["gy"], offsets=none[:1])
    assert (y == 0).all() and (g[0] == 0).all() and (g[1] == 0).all()
    assert gpu.short_conv_step(on["x"][:0], on["w"], torch.zeros(1, 3, 12, device="cuda")).shape == (0, 12)


def test_not_finite_inputs_reach_the_tokens_of_their_window_alone(gpu):
    p, on = make(7, "fp32", 80, 1, 20, 4)
    y, _ = gpu.short_conv_forward(on["x"][None], on["w"])
    on["x"][30, 3], on["x"][50, 4] = float("nan"), float("inf")
    z, _ = gpu.short_conv_forward(on["x"][None], on["w"])
    clean = torch.ones(80, 20, dtype=torch.bool, device="cuda")
    clean[30:34, 3] = clean[50:54, 4] = False
    assert torch.isnan(z[0, 30:34, 3]).all() and torch.equal(z[0][clean], y[0][clean])


def test_equal_bits_on_another_stream_and_replayed(gpu):
    _, tokens, count, offsets = layout([130, 7, 0, 64])
    p, on = make(8, "bf16", tokens, count, 600, 4)

    def work():
        return (*gpu.short_conv_forward(on["x"], on["w"], bias=on["b"], initial_state=on["s"], offsets=offsets),
                *gpu.short_conv_backward(on["x"], on["w"], on["gy"], bias=on["b"], initial_state=on["s"],
                                         grad_final_state=on["gf"], offsets=offsets))

    want = work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = work()
    here = work()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) and torch.equal(u, w) for u, v, w in zip(want, got, here))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    x = on["x"].clone()
    for i in range(3):
        on["x"].copy_(x * (i + 1))
        eager = [t.clone() for t in work()]
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(eager, held))
