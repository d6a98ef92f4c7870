"""The selective scan on the GPU against its recurrence in float64.

Tolerances.  Every output is rounded once to its type (half a step of the value) and is a
sum of products in 32-bit floats before.  What those are off by is counted in roundings,
2^-24 each, of the same sums taken of magnitudes: a state is multiplied and added to once a
token, its decay is an exponential of a rounded product, so a token adds at most 4 roundings
to a state, 4 to a state's gradient, and a gradient has the product of both: 8 for each token
of the longest sequence.  A step is off by |pre| + 10 roundings (the exponential's argument,
the softplus's own), which an exponential decay turns into at most as many of the largest
magnitude, since r exp(-r) < 1.  Sums over states and channels are trees or 64-bit ones; 64
roundings are allowed for them and for what is done once (gates, slopes, exchanges)."""
import numpy as np
import pytest

import sequence_reference as R
from parity_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ROWS = ("x", "dt", "z", "b", "c")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


def roundings(p, rows, softplus):
    pre = np.abs(p["dt"] + (0 if p["dt_bias"] is None else p["dt_bias"])).max(initial=0.0)
    return (64 + 8 * max([n for _, n in rows], default=0) + 10 + pre) * 2.0 ** -24


def near(name, got, want, size, ulps):
    got = got.detach().double().cpu().numpy().reshape(want.shape)
    half = torch.finfo(name[1]).eps / 2
    tiny = 2.0 ** -25 if name[1] == torch.float16 else 2.0 ** -149
    bad = ~(np.abs(got - want) <= half * np.abs(want) + ulps * size + tiny)
    assert not bad.any(), f"{name[0]}: {bad.sum()} of {bad.size} off, worst {np.abs(got - want).max():.3e}"


def inputs(seed, kind, tokens, sequences, channels, groups, state, gated=True, optional=True, softplus=True):
    """(float64 values, the GPU's tensors) of the type's own numbers."""
    gen = np.random.default_rng(seed)
    p = R.scan_inputs(gen, tokens, sequences, channels, groups, state, gated)
    if not softplus:
        p["dt"] = 0.1 * np.abs(p["dt"])
        p["dt_bias"] = 0.05 * np.abs(p["dt_bias"])
    if not optional:
        p["d"] = p["dt_bias"] = None
    on = {}
    for n, v in p.items():
        if v is None:
            on[n] = None
            continue
        t = torch.from_numpy(v).to(TYPES[kind] if n in ROWS else torch.float32)
        p[n], on[n] = t.double().numpy(), t.cuda()
    return gen, p, on


def some(gen, kind, shape):
    t = torch.from_numpy(gen.standard_normal(shape)).to(kind)
    return t.double().numpy(), t.cuda()


SIZES = [  # channels, groups, state, lengths (packed) or (batch, length)
    (1, 1, 1, [1]), (16, 1, 16, [64]), (17, 1, 16, (2, 65)), (48, 3, 4, [3, 0, 130, 1, 64]), (66, 2, 12, [129, 63]),
    (40, 2, 5, (3, 33)), (20, 1, 32, [70, 31, 0]), (35, 1, 64, (1, 40)), (33, 1, 50, [9, 17]), (64, 4, 8, [257, 0, 0, 2]),
    (8, 8, 3, (5, 7)), (130, 1, 16, [1, 1, 1, 300]),
]


def layout(lens):
    if isinstance(lens, tuple):
        return R.spans(batch=lens[0], length=lens[1]), lens[0] * lens[1], lens[0], None
    rows = R.spans(lens)
    ends = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    return rows, sum(lens), len(lens), ends


def shaped(on, lens):
    """The token rows as [B, T, ...] where the sequences are not packed."""
    if not isinstance(lens, tuple):
        return dict(on)
    return {n: t.unflatten(0, lens) if n in (*ROWS, "gy") and t is not None else t for n, t in on.items()}


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("channels,groups,state,lens", SIZES)
def test_forward(gpu, kind, channels, groups, state, lens):
    rows, tokens, count, offsets = layout(lens)
    for gated, optional, first, softplus in ((True, True, True, True), (False, False, False, True), (True, True, True, False)):
        say(f"[scan] forward {kind} {channels} {groups} {state} {lens} {gated} {first} {softplus}")
        _, p, on = inputs(channels + state, kind, tokens, count, channels, groups, state, gated, optional, softplus)
        if not first:
            p["initial"] = np.zeros_like(p["initial"])
        o = shaped(on, lens)
        y, final = gpu.selective_scan_forward(o["x"], o["dt"], o["a"], o["b"], o["c"], d=o["d"], z=o["z"],
                                              dt_bias=o["dt_bias"], initial_state=o["initial"] if first else None,
                                              softplus=softplus, offsets=offsets)
        want, wf, _ = R.scan(p, rows, softplus)
        size, sf, _ = R.scan(p, rows, softplus, size=True)
        ulps = roundings(p, rows, softplus)
        assert y.dtype == TYPES[kind] and y.shape == o["x"].shape and final.dtype == torch.float32
        near(("y", y.dtype), y, want, size, ulps)
        near(("final", final.dtype), final, wf, sf, ulps)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("channels,groups,state,lens", SIZES)
def test_backward(gpu, kind, channels, groups, state, lens):
    rows, tokens, count, offsets = layout(lens)
    for gated, optional, first, softplus in ((True, True, True, True), (False, False, False, True), (True, True, True, False)):
        say(f"[scan] backward {kind} {channels} {groups} {state} {lens} {gated} {first} {softplus}")
        gen, p, on = inputs(channels + state + 1, kind, tokens, count, channels, groups, state, gated, optional, softplus)
        gy, on["gy"] = some(gen, TYPES[kind], (tokens, channels))
        gf, gfinal = some(gen, torch.float32, (count, channels, state))
        if not first:
            p["initial"], gf, gfinal = np.zeros_like(p["initial"]), 0 * gf, None
        o = shaped(on, lens)
        got = gpu.selective_scan_backward(o["x"], o["dt"], o["a"], o["b"], o["c"], o["gy"], d=o["d"], z=o["z"],
                                          dt_bias=o["dt_bias"], initial_state=o["initial"] if first else None,
                                          grad_final_state=gfinal, softplus=softplus, offsets=offsets)
        _, _, want = R.scan(p, rows, softplus, gy, gf)
        _, _, size = R.scan(p, rows, softplus, gy, gf, size=True)
        ulps = roundings(p, rows, softplus)
        for n, t in zip(R.NAMES, got):
            if p[n] is None or (n == "initial" and not first):
                assert t is None, n
                continue
            assert t.dtype == (TYPES[kind] if n in ROWS else torch.float32)
            near((n, t.dtype), t, want[n], size[n], ulps)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("channels,groups,state,batch,pool", [(1, 1, 1, 1, 1), (16, 1, 16, 5, 9), (50, 2, 12, 70, 64), (33, 1, 64, 3, 3),
                                                              (9, 3, 7, 2, 4), (64, 1, 32, 4, 130)])
def test_step(gpu, kind, channels, groups, state, batch, pool):
    for gated in (True, False):
        say(f"[scan] step {kind} {channels} {groups} {state} {batch} {pool} {gated}")
        gen, p, on = inputs(7 * batch + state, kind, batch, pool, channels, groups, state, gated, gated)
        # (with 70 rows of 64 slots some are named twice)
        slots = gen.permutation(np.resize(np.arange(pool), max(batch, pool)))[:batch]
        if batch > 2:
            slots[1], slots[-1] = -1, pool
        want, states = np.zeros((batch, channels)), p["initial"].copy()
        size, ssize, off = np.zeros((batch, channels)), np.abs(states), 0.0
        for b, s in enumerate(slots):
            if not 0 <= s < pool:
                continue
            q = {n: v[b:b + 1] if n in ROWS and v is not None else v for n, v in p.items()}
            one = R.spans([1])
            off = max(off, roundings(q, one, True))
            size[b], ssize[s] = (v[0] for v in R.scan({**q, "initial": ssize[s:s + 1]}, one, size=True)[:2])
            want[b], states[s] = (v[0] for v in R.scan({**q, "initial": states[s:s + 1]}, one)[:2])
        off *= 1 + max(np.bincount(slots[(slots >= 0) & (slots < pool)], minlength=1))
        pool_gpu = on["initial"].clone()
        y = gpu.selective_scan_step(on["x"], on["dt"], on["a"], on["b"], on["c"], pool_gpu,
                                    slots=torch.tensor(slots, dtype=torch.int32).cuda(), d=on["d"], z=on["z"],
                                    dt_bias=on["dt_bias"])
        near(("y", y.dtype), y, want, size, off)
        near(("states", torch.float32), pool_gpu, states, ssize, off)
        left = [s for s in range(pool) if s not in set(slots.tolist())]
        assert torch.equal(pool_gpu[left], on["initial"][left])
        if batch <= pool:
            again = on["initial"].clone()
            y = gpu.selective_scan_step(on["x"], on["dt"], on["a"], on["b"], on["c"], again, d=on["d"], z=on["z"],
                                        dt_bias=on["dt_bias"])
            q = {**p, "initial": p["initial"][:batch]}
            each = R.spans(batch=batch, length=1)
            near(("y", y.dtype), y, R.scan(q, each)[0], R.scan(q, each, size=True)[0], roundings(q, each, True))


def test_slices_strides_and_given_buffers(gpu):
    """Rows of one projection, broadcast groups, rows behind the last sequence, states in place."""
    gen, p, on = inputs(3, "bf16", 90, 3, 24, 2, 16)
    lens, t = [40, 0, 33], torch.bfloat16
    rows, used, _, offsets = layout(lens)
    wide = torch.full((90, 24 * 3 + 2 * 32 + 6), 9.0, device="cuda", dtype=t)
    at, views = 3, {}
    for n in ("x", "dt", "z"):
        views[n] = wide[:, at:at + 24]
        at += 24
    for n in ("b", "c"):
        views[n] = wide[:, at:at + 32].unflatten(-1, (2, 16))
        at += 32
    for n, v in views.items():
        v.copy_(on[n])
    kept = wide.clone()
    call = lambda q, **more: gpu.selective_scan_forward(  # noqa: E731
        q["x"], q["dt"], on["a"], q["b"], q["c"], d=on["d"], z=q["z"], dt_bias=on["dt_bias"], offsets=offsets, **more)
    y, final = call(on, initial_state=on["initial"])
    assert (y[used:] == 0).all()
    given, state = torch.full_like(y, 5.0), on["initial"].clone()
    y2, final2 = call(views, initial_state=state, y=given, final_state=state)
    assert y2 is given and final2 is state
    assert torch.equal(y2[:used], y[:used]) and torch.equal(state, final) and (y2[used:] == 5).all()
    assert torch.equal(state[1], on["initial"][1])  # of no tokens
    gy = on["x"].flip(0).contiguous()
    back = lambda q, g, **more: gpu.selective_scan_backward(  # noqa: E731
        q["x"], q["dt"], on["a"], q["b"], q["c"], g, d=on["d"], z=q["z"], dt_bias=on["dt_bias"], offsets=offsets,
        initial_state=on["initial"], **more)
    gf = torch.randn_like(on["initial"])
    want = back(on, gy, grad_final_state=gf)
    wide2 = torch.cat([gy, gy], 1)
    state = gf.clone()
    rest = torch.full_like(want[3], 7.0)
    got = back(views, wide2[:, 24:], grad_final_state=state, grad_initial_state=state, grad_b=rest)
    for n, u, v in zip(R.NAMES, want, got):
        same = slice(0, used) if n == "b" else slice(None)
        assert torch.equal(u[same], v[same]), n
        if n in ROWS:
            assert (u[used:] == 0).all(), n
    assert (rest[used:] == 7).all() and torch.equal(wide, kept)
    # one b and c for both groups, read at a stride of nothing
    both = {**on, "b": on["b"][:, :1].expand(-1, 2, -1), "c": on["c"][:, :1].expand(-1, 2, -1)}
    one = {**on, "b": on["b"][:, :1].contiguous(), "c": on["c"][:, :1].contiguous()}
    assert torch.equal(call(both)[0], call(one)[0])
    gb, gc = back(both, gy)[3:5]
    wb, wc = back(one, gy)[3:5]
    for two, alone in ((gb, wb), (gc, wc)):
        sum2 = two.float().sum(1)
        room = 2.0 ** -8 * (two.float().abs().sum(1) + alone[:, 0].float().abs()) + 1e-6
        assert ((sum2 - alone[:, 0].float()).abs() <= room).all()


def test_nothing_to_do(gpu):
    _, _, on = inputs(5, "fp32", 0, 2, 8, 1, 4)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    y, final = gpu.selective_scan_forward(on["x"], on["dt"], on["a"], on["b"], on["c"], initial_state=on["initial"], offsets=none)
    assert y.shape == (0, 8) and torch.equal(final, on["initial"])
    gf = torch.randn_like(on["initial"])
    g = gpu.selective_scan_backward(on["x"], on["dt"], on["a"], on["b"], on["c"], on["x"], d=on["d"],
                                    initial_state=on["initial"], grad_final_state=gf, offsets=none)
    assert (g[2] == 0).all() and (g[5] == 0).all() and torch.equal(g[8], gf)
    _, _, on = inputs(5, "fp32", 4, 0, 8, 1, 4)
    y, final = gpu.selective_scan_forward(on["x"], on["dt"], on["a"], on["b"], on["c"], offsets=none[:1])
    assert (y == 0).all() and final.shape == (0, 8, 4)
    g = gpu.selective_scan_backward(on["x"], on["dt"], on["a"], on["b"], on["c"], on["x"], offsets=none[:1])
    assert all((t == 0).all() for t in g if t is not None)
    y = gpu.selective_scan_step(on["x"][:0], on["dt"][:0], on["a"], on["b"][:0], on["c"][:0], torch.zeros(2, 8, 4, device="cuda"))
    assert y.shape == (0, 8)


def test_values_that_are_not_finite_stay_in_their_channel_and_behind(gpu):
    _, _, on = inputs(9, "fp32", 150, 2, 20, 1, 16)
    offsets = torch.tensor([0, 100, 150], dtype=torch.int32, device="cuda")
    call = lambda: gpu.selective_scan_forward(on["x"], on["dt"], on["a"], on["b"], on["c"], d=on["d"], z=on["z"],  # noqa: E731
                                              offsets=offsets)
    y, final = call()
    on["x"][70, 3] = float("nan")
    on["x"][20, 5] = float("inf")
    y2, final2 = call()
    assert torch.isnan(y2[70:100, 3]).all() and not torch.isfinite(y2[20:100, 5]).any()
    assert torch.isnan(final2[0, 3]).all()
    clean = torch.ones_like(y, dtype=torch.bool)
    clean[70:100, 3] = clean[20:100, 5] = False
    assert torch.equal(y2[clean], y[clean]) and torch.equal(final2[1], final[1])


def test_steps_of_nothing_and_of_everything(gpu):
    """softplus far from zero: what is next to nothing keeps its digits, a long step forgets."""
    _, p, on = inputs(10, "fp32", 6, 1, 16, 1, 16)
    dt = torch.tensor([-1e30, -100.0, -20.0, -8.0, 80.0, float("-inf")], device="cuda")[:, None].expand(6, 16).contiguous()
    p["dt"], p["dt_bias"] = dt.double().cpu().numpy(), None
    y, final = gpu.selective_scan_forward(on["x"][None], dt[None], on["a"], on["b"][None], on["c"][None], d=on["d"], z=on["z"][None],
                                          initial_state=on["initial"])
    p["dt"][-1] = -1e30
    rows = R.spans([6])
    ulps = (64 + 48 + 10) * 2.0 ** -24 + 100 * 2.0 ** -24  # of a step at most |pre|, where it counts (-100 and 80)
    near(("y", y.dtype), y, R.scan(p, rows)[0], R.scan(p, rows, size=True)[0], ulps)
    near(("final", final.dtype), final, R.scan(p, rows)[1], R.scan(p, rows, size=True)[1], ulps)


def test_equal_bits_on_another_stream_and_replayed(gpu):
    lens = [130, 7, 64]
    _, tokens, count, offsets = layout(lens)
    _, _, on = inputs(12, "bf16", tokens, count, 40, 2, 16)
    gy, gf = torch.randn_like(on["x"]), torch.randn_like(on["initial"])

    def work():
        y, final = gpu.selective_scan_forward(on["x"], on["dt"], on["a"], on["b"], on["c"], d=on["d"], z=on["z"],
                                              dt_bias=on["dt_bias"], initial_state=on["initial"], offsets=offsets)
        return (y, final, *gpu.selective_scan_backward(on["x"], on["dt"], on["a"], on["b"], on["c"], gy, d=on["d"], z=on["z"],
                                                       dt_bias=on["dt_bias"], initial_state=on["initial"],
                                                       grad_final_state=gf, offsets=offsets))

    want = work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = work()
    here = work()  # at the same time
    side.synchronize()
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


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, a, b, c, d, z, dt_bias, initial):
        import cfc_recurrent_cell_amd as C
        ctx.save_for_backward(x, dt, a, b, c, d, z, dt_bias, initial)
        return C.selective_scan_forward(x, dt, a, b, c, d=d, z=z, dt_bias=dt_bias, initial_state=initial)

    @staticmethod
    def backward(ctx, gy, gf):
        import cfc_recurrent_cell_amd as C
        x, dt, a, b, c, d, z, dt_bias, initial = ctx.saved_tensors
        return C.selective_scan_backward(x, dt, a, b, c, gy.contiguous(), d=d, z=z, dt_bias=dt_bias, initial_state=initial,
                                         grad_final_state=gf.contiguous())


def test_gradients_against_differences(gpu):
    """Along a direction, of the kernels' own outputs: the value v is a sum of 2 * 70 * 16
    products, off by the forward's bound of the size of its terms, and so is each side of the
    difference; with a step s the difference is off by that over s, and by s^2 of the third
    derivative, which is estimated from the float64 reference."""
    _, p, on = inputs(14, "fp32", 70, 1, 16, 1, 16)
    gen = np.random.default_rng(1)
    leaves = {n: (t[None] if n in ROWS else t).clone().requires_grad_() for n, t in on.items()}
    gy, gf = gen.standard_normal((70, 16)), gen.standard_normal((1, 16, 16))
    ty, tf = torch.tensor(gy, device="cuda"), torch.tensor(gf, device="cuda")
    ways = {n: gen.standard_normal(v.shape) * 0.1 for n, v in p.items()}
    y, final = Scan.apply(*(leaves[n] for n in R.NAMES))
    ((y[0].double() * ty).sum() + (final.double() * tf).sum()).backward()
    slope = sum(float((leaves[n].grad.double().cpu().numpy().reshape(ways[n].shape) * ways[n]).sum()) for n in R.NAMES)

    def exact(s):
        q = {n: v + s * ways[n] for n, v in p.items()}
        y, final, _ = R.scan(q, R.spans([70]))
        return (y * gy).sum() + (final * gf).sum()

    def kernel(s):
        q = {n: (p[n] + s * ways[n]) for n in p}
        q = {n: torch.tensor(v, dtype=torch.float32, device="cuda") for n, v in q.items()}
        q = {n: t[None] if n in ROWS else t for n, t in q.items()}
        y, final = gpu.selective_scan_forward(q["x"], q["dt"], q["a"], q["b"], q["c"], d=q["d"], z=q["z"], dt_bias=q["dt_bias"],
                                              initial_state=q["initial"])
        return float((y[0].double() * ty).sum() + (final.double() * tf).sum())

    s = 0.02
    y_size, f_size, _ = R.scan(p, R.spans([70]), size=True)
    size = (y_size * np.abs(gy)).sum() + (f_size * np.abs(gf)).sum()
    noise = roundings(p, R.spans([70]), True) * size / s
    third = abs((exact(s) - exact(-s)) / (2 * s) - (exact(s / 8) - exact(-s / 8)) / (s / 4))
    got = (kernel(s) - kernel(-s)) / (2 * s)
    assert abs(got - slope) <= noise + 2 * third, (got, slope, noise, third)
