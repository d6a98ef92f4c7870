"""The delta rule and the norms run together, as a layer of a model: trained through
autograd over packed sequences, and served, a prompt at once and then token by token
from the pool of states with the step captured.

Tolerances.  Trained, in fp32: each stage may be off by its own bound (64
roundings of 2^-24 of the value for a norm, one for each addition of a product,
dim_k + 3 * 64 of the largest magnitude for the delta rule).  What such errors become
further on is taken from the float64 layer itself: it is run again with every stage's
output off by its whole bound, the signs at random, and four times the largest
change over four such runs is allowed.  Served, each operator is held to float64 of
what it was given, with its own bound: half a step of the type, the roundings above, and
2^-13 of the largest magnitude for a prompt's 16-bit o."""
import numpy as np
import pytest

import delta_rule_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
EPS = 1e-6
LENS, HK, HV, DK, DV, WIDTH = [70, 0, 1, 129], 2, 4, 24, 40, 96


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests selected but torch sees no GPU")
    import cfc_recurrent_cell_amd as C
    C.load_library()
    return C


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual):
        import cfc_recurrent_cell_amd as C
        y, h, rstd = C.rms_norm_forward(x, weight, EPS, residual=residual)
        ctx.save_for_backward(h, weight, rstd)
        ctx.both = residual is not None
        return y, h

    @staticmethod
    def backward(ctx, gy, gh):
        import cfc_recurrent_cell_amd as C
        h, weight, rstd = ctx.saved_tensors
        gx, gw = C.rms_norm_backward(gy.contiguous(), h, weight, rstd, grad_h=gh.contiguous())
        return gx, gw.to(weight.dtype), gx if ctx.both else None


class Delta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, s0, offsets):
        import cfc_recurrent_cell_amd as C
        ctx.save_for_backward(q, k, v, g, beta, s0, offsets)
        return C.delta_rule_forward(q, k, v, g, beta, initial_state=s0, offsets=offsets)

    @staticmethod
    def backward(ctx, go, gfinal):
        import cfc_recurrent_cell_amd as C
        q, k, v, g, beta, s0, offsets = ctx.saved_tensors
        return *C.delta_rule_backward(q, k, v, g, beta, go.contiguous(), initial_state=s0, offsets=offsets,
                                      grad_final_state=gfinal.contiguous()), None


def plain_norm(x, weight, residual):
    h = x if residual is None else x + residual
    return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * weight, h


def plain_delta(q, k, v, g, beta, s0, _):
    k, q = k.repeat_interleave(HV // HK, 1), q.repeat_interleave(HV // HK, 1)
    o, final, at = [], [], 0
    for i, n in enumerate(LENS):
        s = s0[i]
        for t in range(at, at + n):
            s = s * g[t].exp()[:, None, None]
            u = beta[t][:, None] * (v[t] - (s * k[t][:, :, None]).sum(1))
            s = s + k[t][:, :, None] * u[:, None, :]
            o.append(DK ** -0.5 * (s * q[t][:, :, None]).sum(1))
        final.append(s)
        at += n
    return torch.stack(o), torch.stack(final)


def layer(p, norm, delta, offsets, off):
    """The layer's outputs; off(tensor, roundings, of the largest?) is applied to each stage's."""
    y, h = norm(p["x"], p["w_in"], p["residual"])
    y, h = off(y, 64), off(h, 1)
    rows = off(y @ p["w_qkv"], WIDTH)
    q, k, v, a, b = rows.split([HK * DK, HK * DK, HV * DV, HV, HV], -1)
    unit = lambda t: off(torch.nn.functional.normalize(t.unflatten(-1, (HK, DK)), dim=-1), DK + 8)  # noqa: E731
    g = off(-0.1 * torch.nn.functional.softplus(a), 16)
    beta = off(torch.sigmoid(b), 16)
    o, final = delta(unit(q), unit(k), v.unflatten(-1, (HV, DV)), g.contiguous(), beta.contiguous(), p["s0"], offsets)
    o, final = off(o, DK + 192, True), off(final, DK + 192, True)
    z, _ = norm(o, p["w_head"], None)
    z = off(z, 64)
    return off(z.flatten(-2) @ p["w_out"], HV * DV) + h, final


class Off(torch.autograd.Function):
    """Values, and on the way back their gradients, off by so many roundings."""

    @staticmethod
    def forward(ctx, t, n, gen, top):
        ctx.n, ctx.gen, ctx.top = n, gen, top
        return Off.by(t, n, gen, top)

    @staticmethod
    def by(t, n, gen, top):
        sign = torch.randint(0, 2, t.shape, generator=gen).double() * 2 - 1
        size = t.abs().max() if top and t.numel() else t.abs()
        return t + n * 2.0 ** -24 * sign * size

    @staticmethod
    def backward(ctx, g):
        # a gradient of a stage is a sum of as many terms, or is a difference: of the largest
        return Off.by(g, ctx.n, ctx.gen, True), None, None, None


def train(p, norm, delta, offsets, off, aim):
    p = {n: t.detach().clone().requires_grad_() for n, t in p.items()}
    out, final = layer(p, norm, delta, offsets, off)
    ((out * aim[0]).sum() + (final * aim[1]).sum()).backward()
    return {"out": out.detach(), "final": final.detach(), **{"grad " + n: t.grad for n, t in p.items()}}


def test_a_layer_is_trained_over_packed_sequences():
    gen = torch.Generator().manual_seed(11)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    T = sum(LENS)
    p = {"x": n(T, WIDTH), "residual": n(T, WIDTH), "w_in": 1 + 0.2 * n(WIDTH),
         "w_qkv": n(WIDTH, 2 * HK * DK + HV * DV + 2 * HV) * WIDTH ** -0.5, "w_head": 1 + 0.2 * n(DV),
         "w_out": n(HV * DV, WIDTH) * (HV * DV) ** -0.5, "s0": 0.3 * n(len(LENS), HV, DK, DV)}
    aim = [n(T, WIDTH), n(len(LENS), HV, DK, DV)]
    exact = {k: t.double() for k, t in p.items()}
    aim64 = [t.double() for t in aim]
    same = lambda t, *_: t  # noqa: E731
    want = train(exact, plain_norm, plain_delta, None, same, aim64)
    change = {k: 0.0 for k in want}
    for seed in range(4):
        g2 = torch.Generator().manual_seed(seed)
        got = train(exact, plain_norm, plain_delta, None, lambda t, m, top=False: Off.apply(t, m, g2, top), aim64)
        change = {k: max(change[k], float((got[k] - want[k]).abs().max())) for k in want}
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int32).cuda()
    on = {k: t.cuda() for k, t in p.items()}
    got = train(on, Norm.apply, Delta.apply, offsets, same, [t.cuda() for t in aim])
    for k, w in want.items():
        worst = float((got[k].double().cpu() - w).abs().max())
        assert worst <= 4 * change[k], f"{k}: {worst:.3e} off, {4 * change[k]:.3e} allowed"
        assert change[k] < 2e-3 * float(w.abs().max()), k  # the bound says something


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_prompts_then_a_captured_step(gpu, kind):
    C, t, steps = gpu, {"bf16": torch.bfloat16, "fp16": torch.float16}[kind], 5
    lens, pool, width, group = [33, 70, 5], 6, 256, 64
    slots = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    w_in, w_head = (1 + 0.2 * n(width)).to(t), (1 + 0.2 * n(DV)).to(t)
    w = n(width, 2 * HK * DK + HV * DV + 2 * HV) * width ** -0.5
    half = torch.finfo(t).eps / 2
    tiny = 2.0 ** -25 if kind == "fp16" else 0.0

    def inner(y):
        q, k, v, a, b = (y @ w).split([HK * DK, HK * DK, HV * DV, HV, HV], -1)
        unit = lambda m: torch.nn.functional.normalize(m.unflatten(-1, (HK, DK)), dim=-1).to(t)  # noqa: E731
        return (unit(q), unit(k), v.unflatten(-1, (HV, DV)).to(t), -0.1 * torch.nn.functional.softplus(a),
                torch.sigmoid(b))

    def norm_near(o, z):
        o = o.double()
        want = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * w_head.double()
        assert bool(((z.double() - want).abs() <= half * want.abs() + 64 * 2.0 ** -24 * want.abs() + tiny).all())

    # the prompts, packed; their last states go to the pool
    y, _, _ = C.rms_norm_forward(n(sum(lens), width).to(t), w_in, EPS, want_rstd=False)
    prompt = inner(y.float())
    offsets = torch.tensor([0, 33, 103, 108], dtype=torch.int32).cuda()
    o, final = C.delta_rule_forward(*prompt, offsets=offsets)
    norm_near(o, C.rms_norm_forward(o, w_head, EPS)[0])
    states = torch.full((pool, HV, DK, DV), 7.0, device="cuda")
    states[slots.long()] = final

    # a step: the 8-bit norm, its product, the states, the heads' norm
    x, stream = torch.zeros(3, width, device="cuda", dtype=t), torch.zeros(3, width, device="cuda", dtype=t)

    def step():
        y8, scales, _ = C.rms_norm_forward_e4m3(x, w_in, EPS, residual=stream, h=stream, group=group)
        row = inner((y8.float().unflatten(-1, (-1, group)) * scales[..., None]).flatten(-2))
        o = C.delta_rule_step(*row, states, slots)
        return y8, scales, row, o, C.rms_norm_forward(o, w_head, EPS)[0]

    xs, start = n(steps, 3, width).to(t), n(3, width).to(t)
    kept = states.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()

    def run(one):
        states.copy_(kept)
        stream.copy_(start)
        got, h = [], start.clone()
        for i in range(steps):
            x.copy_(xs[i])
            y8, scales, row, o, z = one()
            torch.cuda.synchronize()
            h = (h.float() + xs[i].float()).to(t)
            assert torch.equal(stream, h)
            want = plain_norm(h.double(), w_in.double(), None)[0]
            top = want.unflatten(-1, (-1, group)).abs().amax(-1)
            assert bool(((scales.double() - top / 448).abs() <= 68 * 2.0 ** -24 * top / 448).all())
            each = scales.double()[..., None]
            parts = want.unflatten(-1, (-1, group))
            back = y8.double().unflatten(-1, (-1, group)) * each
            allowed = 2.0 ** -4 * parts.abs() + 2.0 ** -10 * each + 132 * 2.0 ** -24 * parts.abs()
            assert bool(((back - parts).abs() <= allowed).all())
            norm_near(o, z)
            got.append([m.clone() for m in (*row, o)])
        return got, states.clone()

    def replayed():
        graph.replay()
        return outs

    eager, eager_states = run(step)
    for _ in range(3):
        again, again_states = run(replayed)
        assert torch.equal(again_states, eager_states)
        assert all(torch.equal(a, b) for one, two in zip(again, eager) for a, b in zip(one, two))
        (n(300, 300) @ n(300, 300)).sum().item()
    assert torch.equal(eager_states[[1, 3, 5]], kept[[1, 3, 5]])

    # prompt and steps of each sequence as one, in float64
    at = 0
    for i, m in enumerate(lens):
        seq = [torch.cat([p[at:at + m], torch.stack([r[j][i] for r in eager])]).double().cpu().numpy()
               for j, p in enumerate(prompt)]
        want, last, _ = R.forward(*seq, np.zeros((1, HV, DK, DV)), DK ** -0.5, [(0, m + steps)])
        got = torch.cat([o[at:at + m], torch.stack([r[5][i] for r in eager])]).double().cpu().numpy()
        more = (DK + 192) * 2.0 ** -24
        top = np.abs(want).max()
        assert (np.abs(got - want) <= half * np.abs(want) + (more + 2.0 ** -13) * top + tiny).all()
        state = eager_states[int(slots[i])].double().cpu().numpy()
        assert (np.abs(state - last[0]) <= 2.0 ** -24 * np.abs(last[0]) + more * np.abs(last).max()).all()
        at += m
