"""The layer norm, the short convolution, the selective scan and the clipping of gradients run
together, as a layer of a model: trained through autograd over packed sequences with its
gradients clipped, and served, prompts at once and then token by token from pools of states
with the step captured.

Tolerances.  Trained, in fp32: each stage may be off by its own bound (64 roundings of 2^-24
of the value for a norm, 16 of the largest magnitude for the convolution, 64 + 8 a token of
the longest sequence for the scan, one for each addition of a product).  What such errors
become further on is taken from the float64 layer itself: it is run again with every stage's
output off by its whole bound, the signs at random, and four times the largest change over
four such runs is allowed.  Served, each operator is held to float64 of what it was given,
with its own bound."""
import numpy as np
import pytest

import sequence_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
EPS = 1e-5
LENS, WIDTH, CH, GROUPS, STATE, TAPS, LOW = [70, 0, 1, 129], 48, 40, 2, 6, 4, 5
ULP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual):
        import cfc_recurrent_cell_amd as C
        y, h, mean, rstd = C.layer_norm_forward(x, weight, bias, EPS, residual=residual)
        ctx.save_for_backward(h, weight, mean, rstd)
        return y, h

    @staticmethod
    def backward(ctx, gy, gh):
        import cfc_recurrent_cell_amd as C
        h, weight, mean, rstd = ctx.saved_tensors
        gx, gw, gb = C.layer_norm_backward(gy.contiguous(), h, weight, mean, rstd, grad_h=gh.contiguous())
        return gx, gw, gb, gx


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial, offsets):
        import cfc_recurrent_cell_amd as C
        ctx.save_for_backward(x, weight, bias, initial, offsets)
        return C.short_conv_forward(x, weight, bias=bias, initial_state=initial, offsets=offsets)

    @staticmethod
    def backward(ctx, gy, gf):
        import cfc_recurrent_cell_amd as C
        x, weight, bias, initial, offsets = ctx.saved_tensors
        gx, gw, gb, gi = C.short_conv_backward(x, weight, gy.contiguous(), bias=bias, initial_state=initial,
                                               grad_final_state=gf.contiguous(), offsets=offsets)
        return gx, gw, gb, gi, None


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, a, b, c, d, z, dt_bias, initial, offsets):
        import cfc_recurrent_cell_amd as C
        ctx.save_for_backward(x, dt, a, b, c, d, z, dt_bias, initial, offsets)
        return C.selective_scan_forward(x, dt, a, b, c, d=d, z=z, dt_bias=dt_bias, initial_state=initial, offsets=offsets)

    @staticmethod
    def backward(ctx, gy, gf):
        import cfc_recurrent_cell_amd as C
        x, dt, a, b, c, d, z, dt_bias, initial, offsets = ctx.saved_tensors
        return (*C.selective_scan_backward(x, dt, a, b, c, gy.contiguous(), d=d, z=z, dt_bias=dt_bias, initial_state=initial,
                                           grad_final_state=gf.contiguous(), offsets=offsets), None)


# The same in float64 through torch's own autograd.
def plain_norm(x, weight, bias, residual):
    h = x + residual
    away = h - h.mean(-1, keepdim=True)
    return away * torch.rsqrt(away.square().mean(-1, keepdim=True) + EPS) * weight + bias, h


def pieces(offsets, *rows):
    at = 0
    for i, n in enumerate(LENS):
        yield (i, *(None if t is None else t[at:at + n] for t in rows))
        at += n


def plain_conv(x, weight, bias, initial, offsets):
    ys, finals = [], []
    for i, part in pieces(offsets, x):
        seen = torch.cat([initial[i], part])
        p = sum(seen[j:j + len(part)] * weight[:, j] for j in range(TAPS)) + bias
        ys.append(p * torch.sigmoid(p))
        finals.append(seen[len(part):])
    return torch.cat(ys), torch.stack(finals)


def plain_scan(x, dt, a, b, c, d, z, dt_bias, initial, offsets):
    ys, finals = [], []
    share = CH // GROUPS
    for i, xs, dts, bs, cs, zs in pieces(offsets, x, dt, b, c, z):
        h = initial[i]
        for t in range(len(xs)):
            step = torch.nn.functional.softplus(dts[t] + dt_bias)
            bt, ct = (m[t].repeat_interleave(share, 0) for m in (bs, cs))
            h = torch.exp(step[:, None] * a) * h + (step * xs[t])[:, None] * bt
            ys.append(((h * ct).sum(-1) + d * xs[t]) * zs[t] * torch.sigmoid(zs[t]))
        finals.append(h)
    return torch.stack(ys), torch.stack(finals)


def layer(p, norm, conv, scan, offsets, off):
    y, h = norm(p["x"], p["w_norm"], p["b_norm"], p["residual"])
    y = off(y, 64)
    xz = off(y @ p["w_in"], WIDTH)
    x, z = xz[:, :CH], xz[:, CH:]
    x, kept = conv(x, p["w_conv"], p["b_conv"], p["c0"], offsets)
    x = off(x, 16, True)
    low = off(x @ p["w_low"], CH)
    dt = off(low[:, :LOW] @ p["w_dt"], LOW)
    b, c = (t.unflatten(-1, (GROUPS, STATE)) for t in low[:, LOW:].split([GROUPS * STATE] * 2, -1))
    o, final = scan(x, dt, -torch.exp(p["log_a"]), b, c, p["d"], z, p["dt_bias"], p["s0"], offsets)
    n = 64 + 8 * max(LENS)
    o, final = off(o, n, True), off(final, n, True)
    return off(o @ p["w_out"], CH) + h, kept, final


class Off(torch.autograd.Function):
    """Values, and on the way back their gradients, off by so many roundings."""

    @staticmethod
    def forward(ctx, t, n, gen, top):
        ctx.n, ctx.gen = n, gen
        return Off.by(t, n, gen, top)

    @staticmethod
    def by(t, n, gen, top):
        sign = torch.randint(0, 2, t.shape, generator=gen).double() * 2 - 1
        size = t.abs().max() if top and t.numel() else t.abs()
        return t + n * ULP * sign * size

    @staticmethod
    def backward(ctx, g):
        return Off.by(g, ctx.n, ctx.gen, True), None, None, None


def train(p, norm, conv, scan, offsets, off, aim):
    p = {n: t.detach().clone().requires_grad_() for n, t in p.items()}
    outs = layer(p, norm, conv, scan, offsets, off)
    sum((o * w).sum() for o, w in zip(outs, aim)).backward()
    return dict(zip(("out", "kept", "final"), (o.detach() for o in outs))), {n: t.grad for n, t in p.items()}


def parameters(n):
    T, S = sum(LENS), len(LENS)
    p = {"x": n(T, WIDTH), "residual": n(T, WIDTH), "w_norm": 1 + 0.2 * n(WIDTH), "b_norm": 0.2 * n(WIDTH),
         "w_in": n(WIDTH, 2 * CH) * WIDTH ** -0.5, "w_conv": 0.5 * n(CH, TAPS), "b_conv": 0.1 * n(CH),
         "c0": n(S, TAPS - 1, CH), "w_low": n(CH, LOW + 2 * GROUPS * STATE) * CH ** -0.5, "w_dt": n(LOW, CH) * LOW ** -0.5,
         "log_a": n(CH, STATE), "d": 1 + 0.2 * n(CH), "dt_bias": n(CH) - 2, "s0": 0.3 * n(S, CH, STATE),
         "w_out": n(CH, WIDTH) * CH ** -0.5}
    return p, [n(T, WIDTH), n(S, TAPS - 1, CH), n(S, CH, STATE)]


def test_a_layer_is_trained_over_packed_sequences_with_clipped_gradients(gpu):
    gen = torch.Generator().manual_seed(17)
    p, aim = parameters(lambda *s: torch.randn(*s, generator=gen))
    exact, aim64 = {k: t.double() for k, t in p.items()}, [t.double() for t in aim]
    same = lambda t, *_: t  # noqa: E731
    plain = (plain_norm, plain_conv, plain_scan)
    values, grads = train(exact, *plain, None, same, aim64)
    want = {**values, **{"grad " + k: g for k, g in grads.items()}}
    change = {k: 0.0 for k in want}
    for seed in range(4):
        g2 = torch.Generator().manual_seed(seed)
        v, g = train(exact, *plain, None, lambda t, m, top=False: Off.apply(t, m, g2, top), aim64)
        for k, t in {**v, **{"grad " + k: t for k, t in g.items()}}.items():
            change[k] = max(change[k], float((t - want[k]).abs().max()))
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int32).cuda()
    on = {k: t.cuda() for k, t in p.items()}
    values, grads = train(on, Norm.apply, Conv.apply, Scan.apply, offsets, same, [t.cuda() for t in aim])
    for k, got in {**values, **{"grad " + k: g for k, g in grads.items()}}.items():
        worst = float((got.double().cpu() - want[k]).abs().max())
        assert worst <= 4 * change[k], f"{k}: {worst:.3e} off, {4 * change[k]:.3e} allowed"
        assert change[k] < 5e-3 * float(want[k].abs().max()), k  # the bound says something

    # the gradients of what the layer learns, clipped to half their norm
    learned = [k for k in p if k not in ("x", "residual", "c0", "s0")]
    kept = [grads[k].clone() for k in learned]
    whole = float(torch.cat([g.double().flatten() for g in kept]).norm())
    norm = gpu.clip_grad_norm([grads[k] for k in learned], 0.5 * whole)
    assert abs(float(norm) - whole) <= 2.0 ** -23 * whole
    factor = 0.5 * whole / (whole + 1e-6)
    for k, g in zip(learned, kept):
        assert ((grads[k].double() - g.double() * factor).abs() <= 4 * ULP * g.double().abs()).all(), k


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_prompts_then_a_captured_step(gpu, kind):
    t, steps, lens, pool = {"bf16": torch.bfloat16, "fp16": torch.float16}[kind], 5, [33, 70, 5], 6
    half, tiny = torch.finfo(t).eps / 2, 2.0 ** -25 if kind == "fp16" else 2.0 ** -149
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    slots = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()
    w_norm, b_norm, w_conv, b_conv = (1 + 0.2 * n(WIDTH)).to(t), (0.2 * n(WIDTH)).to(t), (0.5 * n(CH, TAPS)).to(t), (0.1 * n(CH)).to(t)
    w_in, w_low, w_dt = n(WIDTH, 2 * CH) * WIDTH ** -0.5, n(CH, LOW + 2 * GROUPS * STATE) * CH ** -0.5, n(LOW, CH) * LOW ** -0.5
    a, d, bias = -torch.exp(n(CH, STATE)), 1 + 0.2 * n(CH), n(CH) - 2

    def low_of(x):
        low = x.float() @ w_low
        b, c = (m.unflatten(-1, (GROUPS, STATE)).to(t) for m in low[:, LOW:].split([GROUPS * STATE] * 2, -1))
        return (low[:, :LOW] @ w_dt).to(t), b, c

    # the prompts, packed; their last states go to the pools
    offsets = torch.tensor([0, 33, 103, 108], dtype=torch.int32).cuda()
    y, _, _, _ = gpu.layer_norm_forward(n(sum(lens), WIDTH).to(t), w_norm, b_norm, EPS, want_stats=False)
    xz = (y.float() @ w_in).to(t)
    x, kept = gpu.short_conv_forward(xz[:, :CH], w_conv, bias=b_conv, offsets=offsets)
    dt, b, c = low_of(x)
    o, final = gpu.selective_scan_forward(x, dt, a, b, c, d=d, z=xz[:, CH:], dt_bias=bias, offsets=offsets)
    rows = [[xz[:, :CH], x, dt, b, c, xz[:, CH:], o]]
    conv_pool = torch.full((pool, TAPS - 1, CH), 7.0, device="cuda", dtype=t)
    scan_pool = torch.full((pool, CH, STATE), 7.0, device="cuda")
    conv_pool[slots.long()], scan_pool[slots.long()] = kept, final

    token = torch.zeros(3, WIDTH, device="cuda", dtype=t)
    stream = torch.zeros(3, WIDTH, device="cuda", dtype=t)

    def step():
        y, _, _, _ = gpu.layer_norm_forward(token, w_norm, b_norm, EPS, residual=stream, h=stream, want_stats=False)
        xz = (y.float() @ w_in).to(t)
        x = gpu.short_conv_step(xz[:, :CH], w_conv, conv_pool, slots, bias=b_conv)
        dt, b, c = low_of(x)
        o = gpu.selective_scan_step(x, dt, a, b, c, scan_pool, slots, d=d, z=xz[:, CH:], dt_bias=bias)
        return [y, xz[:, :CH], x, dt, b, c, xz[:, CH:], o]

    tokens, start = n(steps, 3, WIDTH).to(t), n(3, WIDTH).to(t)
    kept = conv_pool.clone(), scan_pool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()

    def run(one):
        conv_pool.copy_(kept[0])
        scan_pool.copy_(kept[1])
        stream.copy_(start)
        got, h = [], start.clone()
        for i in range(steps):
            token.copy_(tokens[i])
            row = one()
            torch.cuda.synchronize()
            h = (h.float() + tokens[i].float()).to(t)
            assert torch.equal(stream, h)
            away = h.double() - h.double().mean(-1, keepdim=True)
            want = away * torch.rsqrt(away.square().mean(-1, keepdim=True) + EPS) * w_norm.double() + b_norm.double()
            room = half * want.abs() + 64 * ULP * (h.double().abs().amax(-1, keepdim=True) * 4 + want.abs()) + tiny
            assert ((row[0].double() - want).abs() <= room).all()
            got.append([m.clone() for m in row[1:]])
        return got, conv_pool.clone(), scan_pool.clone()

    def replayed():
        graph.replay()
        return outs

    eager, eager_conv, eager_scan = run(step)
    for _ in range(3):
        again, again_conv, again_scan = run(replayed)
        assert torch.equal(again_conv, eager_conv) and torch.equal(again_scan, eager_scan)
        assert all(torch.equal(u, v) for one, two in zip(again, eager) for u, v in zip(one, two))
        (n(300, 300) @ n(300, 300)).sum().item()
    others = [1, 3, 5]
    assert torch.equal(eager_conv[others], kept[0][others]) and torch.equal(eager_scan[others], kept[1][others])

    # prompt and steps of each sequence as one, in float64
    at = 0
    for i, m in enumerate(lens):
        raw, xs, dts, bs, cs, zs, os = (np.concatenate([p[at:at + m].double().cpu().numpy(),
                                                        *(r[j][i:i + 1].double().cpu().numpy() for r in eager)])
                                        for j, p in enumerate(rows[0]))
        one = R.spans([m + steps])
        w64, b64 = w_conv.double().cpu().numpy(), b_conv.double().cpu().numpy()
        zero = np.zeros((1, TAPS - 1, CH))
        want, last, _ = R.conv(raw, w64, b64, zero, one)
        size, _, _ = R.conv(raw, w64, b64, zero, one, size=True)
        assert (np.abs(xs - want) <= half * np.abs(want) + 16 * ULP * size + tiny).all()
        np.testing.assert_array_equal(eager_conv[int(slots[i])].double().cpu().numpy(), last[0])
        p = {"x": xs, "dt": dts, "a": a.double().cpu().numpy(), "b": bs, "c": cs, "d": d.double().cpu().numpy(), "z": zs,
             "dt_bias": bias.double().cpu().numpy(), "initial": np.zeros((1, CH, STATE))}
        want, last, _ = R.scan(p, one)
        size, sl, _ = R.scan(p, one, size=True)
        more = (64 + 8 * (m + steps) + 10 + np.abs(p["dt"] + p["dt_bias"]).max()) * ULP
        assert (np.abs(os - want) <= half * np.abs(want) + more * size + tiny).all()
        assert (np.abs(eager_scan[int(slots[i])].double().cpu().numpy() - last[0]) <= ULP * np.abs(last[0]) + more * sl[0]).all()
        at += m
