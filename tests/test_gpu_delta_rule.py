"""The gated delta rule on the GPU against the token-by-token float64 reference.

Tolerances, for a result r of a 32-bit computation rounded to type t once:

    |got - r| <= eps_t / 2 |r| + terms * 2^-24 * size

where `terms` counts the additions that a value passes through in a chunk (a sum
over dim_k, the triangular inverse's and two sums over the chunk's 64 tokens) and
`size` is what they are of: the result's largest magnitude, since no partial sum
of unit keys and gates in (0, 1) is much above it; for grad_g, which is a
difference of sums, the magnitudes' sum that the reference gives.  Products of 16-bit
o's second half (M U) keep 16 bits of each factor: 64 terms of 2^-16 at most, of
random sign, so sqrt(64) 2^-16 = 2^-13 of the largest magnitude."""
import numpy as np
import pytest

import delta_rule_reference as R
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
    return torch.device("cuda:0")


class Case:
    """Inputs in a type, on the GPU (strided if asked) and as float64 of the same values."""

    def __init__(self, seed, kind, lens=None, batch=None, length=None, hk=1, hv=1, dk=128, dv=128, state=True,
                 fused=False, extra=0, **more):
        self.rows = R.spans(lens, batch, length)
        self.tokens = sum(n for _, n in self.rows)
        self.kind, self.t = kind, TYPES[kind]
        x = R.inputs(seed, self.rows, self.tokens, hk, hv, dk, dv, state, **more)
        for n in ("q", "k", "v", "go"):
            x[n] = torch.from_numpy(x[n]).to(self.t).double().numpy()
        self.x, self.state = x, state
        self.scale = dk ** -0.5
        self.dims = (hk, hv, dk, dv)
        lead = (self.tokens + extra,) if lens is not None else (batch, length)
        self.lead = lead

        def dev(a, t=torch.float32):
            a = torch.from_numpy(a)
            if extra:
                a = torch.cat([a, torch.zeros(extra, *a.shape[1:], dtype=a.dtype)])
            return a.to(t).cuda().reshape(*lead, *a.shape[1:])

        self.d = {n: dev(x[n], self.t) for n in ("q", "k", "v", "go")}
        if fused:
            row = torch.cat([self.d[n].flatten(-2) for n in ("q", "k", "v")], -1)
            parts = row.split([hk * dk, hk * dk, hv * dv], -1)
            for n, p, w in zip(("q", "k", "v"), parts, (dk, dk, dv)):
                self.d[n] = p.unflatten(-1, (-1, w))
        self.d["g"], self.d["beta"] = dev(x["g"]), dev(x["beta"])
        self.d["s0"] = torch.from_numpy(x["s0"]).float().cuda() if state else None
        self.d["gfinal"] = torch.from_numpy(x["gfinal"]).float().cuda() if state else None
        self.offsets = None
        if lens is not None:
            self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()

    def args(self):
        return [self.d[n] for n in ("q", "k", "v", "g", "beta")]

    def forward(self, **more):
        import cfc_recurrent_cell_amd as C
        return C.delta_rule_forward(*self.args(), initial_state=self.d["s0"], offsets=self.offsets, **more)

    def backward(self, **more):
        import cfc_recurrent_cell_amd as C
        return C.delta_rule_backward(*self.args(), self.d["go"], initial_state=self.d["s0"],
                                     grad_final_state=self.d["gfinal"], offsets=self.offsets, **more)

    def want_forward(self):
        x = self.x
        return R.forward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], self.scale, self.rows)[:2]

    def want_backward(self):
        x = self.x
        return R.backward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], self.scale, self.rows, x["go"],
                          x["gfinal"])

    def near(self, got, want, name, size=None, more=0.0):
        got = got.double().cpu().numpy().reshape(-1, *want.shape[1:])[:len(want)]
        assert got.shape == want.shape, name
        eps = torch.finfo(self.t).eps / 2 if name in ("o", "q", "k", "v") else 2.0 ** -24
        top = np.abs(want).max() if want.size else 0.0
        size = top if size is None else size
        terms = self.dims[2] + 3 * 64
        tol = eps * np.abs(want) + terms * 2.0 ** -24 * size + more * top
        if name in ("o", "q", "k", "v") and self.kind == "fp16":
            tol = tol + 2.0 ** -25  # fp16 below its normal range has steps of 2^-24
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} off, the worst "
                               f"{np.abs(got - want).max():.3e} of {top:.3e}")

    def check_forward(self, o, final):
        want_o, want_s = self.want_forward()
        self.near(o, want_o, "o", more=0.0 if self.kind == "fp32" else 2.0 ** -13)
        self.near(final, want_s, "final")

    def check_backward(self, grads):
        want, mag = self.want_backward()
        names = ("q", "k", "v", "g", "beta", "initial")
        assert (grads[5] is None) == (self.d["s0"] is None)
        for n, t in zip(names, grads):
            if t is not None:
                self.near(t, want[n], n, size=mag.max() if n in ("g", "beta") and mag.size else None)


LENS = [1, 64, 0, 63, 65, 17, 128, 3, 130, 0]
SHAPES = [  # hk, hv, dk, dv
    (1, 1, 128, 128), (2, 4, 64, 64), (1, 3, 16, 16), (3, 3, 33, 17), (1, 2, 127, 130), (2, 2, 128, 256), (1, 1, 1, 1),
    (1, 1, 65, 5), (4, 4, 96, 80),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("hk,hv,dk,dv", SHAPES)
def test_forward_packed(kind, hk, hv, dk, dv):
    say(f"[delta] forward packed {kind} {hk} {hv} {dk} {dv}")
    c = Case(11, kind, lens=LENS, hk=hk, hv=hv, dk=dk, dv=dv)
    c.check_forward(*c.forward())


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("hk,hv,dk,dv", SHAPES)
def test_backward_packed(kind, hk, hv, dk, dv):
    say(f"[delta] backward packed {kind} {hk} {hv} {dk} {dv}")
    c = Case(12, kind, lens=LENS, hk=hk, hv=hv, dk=dk, dv=dv)
    c.check_backward(c.backward())


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 200])
@pytest.mark.parametrize("state", [False, True])
def test_lengths_dense(length, state):
    say(f"[delta] dense length {length} state {state}")
    c = Case(13 + length, "bf16", batch=3, length=length, hk=2, hv=2, dk=64, dv=48, state=state)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("length", [8, 9, 31, 32, 33])
def test_token_by_token_up_to_32_with_many_heads(kind, length):
    """With 384 heads' states the token kernel takes 32 tokens and the chunks 33; of one head 8 and 9."""
    for batch, hv, dims in ((8, 48, (16, 8)), (1, 1, (100, 36)), (96, 4, (30, 5))):
        say(f"[delta] short {kind} {length} x {batch} x {hv}")
        c = Case(14 + length, kind, batch=batch, length=length, hk=hv // 2 or 1, hv=hv, dk=dims[0], dv=dims[1])
        c.check_forward(*c.forward())


@pytest.mark.parametrize("kind,dk,dv", [("bf16", 64, 64), ("fp16", 40, 24), ("fp32", 128, 36), ("bf16", 33, 7)])
def test_slices_of_one_projection(kind, dk, dv):
    """q, k and v as slices (strided, at odd sizes not aligned) give the bits that contiguous ones give."""
    for packed in (False, True):
        sizes = dict(lens=[70, 5, 64]) if packed else dict(batch=2, length=70)
        a = Case(21, kind, hk=2, hv=4, dk=dk, dv=dv, fused=True, **sizes)
        b = Case(21, kind, hk=2, hv=4, dk=dk, dv=dv, **sizes)
        assert not a.d["q"].is_contiguous()
        for x, y in zip((*a.forward(), *a.backward()), (*b.forward(), *b.backward())):
            assert torch.equal(x, y)
        a.check_forward(*a.forward())


def test_a_head_broadcast_to_all():
    """Strides of zero: one key read by every head."""
    c = Case(22, "bf16", batch=2, length=80, hk=4, hv=4, dk=64, dv=32)
    k0 = c.d["k"][:, :, :1]
    c.d["k"] = k0.expand(-1, -1, 4, -1)
    got = c.forward()
    c.d["k"] = c.d["k"].contiguous()
    for x, y in zip(got, c.forward()):
        assert torch.equal(x, y)


def test_strided_gradient_of_o():
    c = Case(23, "bf16", batch=2, length=70, hk=1, hv=2, dk=64, dv=40)
    want = c.backward()
    wide = torch.zeros(2, 70, 2, 80, dtype=c.t, device="cuda")
    wide[..., 40:] = c.d["go"]
    c.d["go"] = wide[..., 40:]
    for x, y in zip(c.backward(), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("length", [9, 150])
def test_decays_of_all_sizes(length):
    """No decay, decays whose sums leave 32 bits nothing, and total ones."""
    c = Case(24, "fp32", batch=2, length=length, hk=1, hv=3, dk=32, dv=32)
    r = np.random.default_rng(1)
    g = c.x["g"]
    pick = r.integers(0, 6, g.shape)
    g[pick == 0] = 0.0
    g[pick == 1] = -300.0
    g[(pick == 2) & (r.random(g.shape) < 0.3)] = -np.inf
    c.d["g"] = torch.from_numpy(g).float().cuda().reshape(c.d["g"].shape)
    c.check_forward(*c.forward())
    for t in c.backward():
        assert torch.isfinite(t).all()
    g[np.isneginf(g)] = -1e4  # the reference's adjoint takes 0 * inf for these
    c.check_backward(c.backward())


def test_keys_that_repeat():
    """The same unit key again and again: the inverse's entries do not decay."""
    c = Case(25, "fp32", batch=1, length=128, hk=1, hv=1, dk=16, dv=16, rate=0.0)
    c.x["k"][:] = c.x["k"][:1]
    c.d["k"] = torch.from_numpy(c.x["k"]).float().cuda().reshape(c.d["k"].shape)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("beta_top", [0.0, 1.0])
def test_gates_of_zero_and_one(beta_top):
    c = Case(26, "bf16", lens=[100], hk=1, hv=2, dk=64, dv=64)
    c.x["beta"][:] = beta_top
    c.d["beta"].fill_(beta_top)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


def test_rows_behind_the_last_sequence_stay():
    c = Case(27, "bf16", lens=[70, 3], hk=1, hv=2, dk=32, dv=32, extra=40)
    o = torch.full_like(c.d["v"], 7.0)
    c.check_forward(*c.forward(o=o))
    assert (o[73:] == 7.0).all()
    bufs = {n: torch.full_like(c.d[m], 7.0) for n, m in (("grad_q", "q"), ("grad_k", "k"), ("grad_v", "v"),
                                                         ("grad_g", "g"), ("grad_beta", "beta"))}
    c.check_backward(c.backward(**bufs))
    for t in bufs.values():
        assert (t[73:] == 7.0).all()
    short = Case(28, "bf16", lens=[3, 2], hk=1, hv=2, dk=32, dv=32, extra=4)  # the token kernel
    o = torch.full_like(short.d["v"], 7.0)
    short.check_forward(*short.forward(o=o))
    assert (o[5:] == 7.0).all()


def test_no_tokens_and_no_sequences():
    import cfc_recurrent_cell_amd as C
    c = Case(29, "bf16", lens=[0, 0], hk=1, hv=2, dk=32, dv=32)
    o, final = c.forward()
    assert o.shape[0] == 0 and torch.equal(final, c.d["s0"])
    assert torch.equal(c.backward()[5], c.d["gfinal"])
    none = torch.zeros(0, 5, 1, 8, device="cuda")
    gate = torch.zeros(0, 5, 1, device="cuda")
    o, final = C.delta_rule_forward(none, none, none, gate, gate)
    assert o.shape == none.shape and final.shape == (0, 1, 8, 8)


def test_state_updated_where_it_is():
    for length in (5, 90):
        c = Case(30, "bf16", batch=2, length=length, hk=1, hv=2, dk=64, dv=64)
        o, final = c.forward()
        s = c.d["s0"].clone()
        import cfc_recurrent_cell_amd as C
        o2, s2 = C.delta_rule_forward(*c.args(), initial_state=s, final_state=s)
        assert s2 is s and torch.equal(s, final) and torch.equal(o, o2)


def test_split_in_two_calls_is_one_call():
    """A prompt in two calls, the state carried between them: the same up to the chunks' rounding."""
    c = Case(31, "fp32", batch=1, length=150, hk=1, hv=2, dk=64, dv=64)
    import cfc_recurrent_cell_amd as C
    first = [t[:, :90] for t in c.args()[:3]] + [t[:, :90].contiguous() for t in c.args()[3:]]
    rest = [t[:, 90:] for t in c.args()[:3]] + [t[:, 90:].contiguous() for t in c.args()[3:]]
    o1, s = C.delta_rule_forward(*first, initial_state=c.d["s0"])
    o2, s = C.delta_rule_forward(*rest, initial_state=s)
    c.check_forward(torch.cat([o1, o2], 1), s)


# ------------------------------------------------------------------- a token each
def step_case(seed, kind, batch, pool, hk, hv, dk, dv, slots):
    c = Case(seed, kind, batch=batch, length=1, hk=hk, hv=hv, dk=dk, dv=dv)
    r = np.random.default_rng(seed)
    states = (0.3 * r.standard_normal((pool, hv, dk, dv))).astype(np.float32)
    args = [t[:, 0].contiguous() for t in c.args()]
    return c, args, states, None if slots is None else torch.tensor(slots, dtype=torch.int32).cuda()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("hk,hv,dk,dv", SHAPES)
@pytest.mark.parametrize("slots", [None, [4, 0, -1, 2, 0, 7, 0, 9, 4]])
def test_step(kind, hk, hv, dk, dv, slots):
    """In order, and with idle rows and slots named more than once."""
    import cfc_recurrent_cell_amd as C
    say(f"[delta] step {kind} {hk} {hv} {dk} {dv} {slots}")
    batch, pool = 9, 9
    c, args, states, sl = step_case(41, kind, batch, pool, hk, hv, dk, dv, slots)
    s = torch.from_numpy(states).cuda()
    o = C.delta_rule_step(*args, s, slots=sl)
    want_s, want_o = states.astype(np.float64), np.zeros((batch, hv, dv))
    x = c.x
    for b, at in enumerate(slots or range(batch)):
        if 0 <= at < pool:
            one = slice(b, b + 1)
            got, fin, _ = R.forward(x["q"][one], x["k"][one], x["v"][one], x["g"][one], x["beta"][one],
                                    want_s[at:at + 1], c.scale, [(0, 1)])
            want_o[b], want_s[at] = got[0], fin[0]
    c.near(o, want_o, "o")
    c.near(s, want_s, "states")
    for at in set(range(pool)) - set(slots or range(pool)):
        assert torch.equal(s[at].cpu(), torch.from_numpy(states[at]))
    if slots:
        assert (o[2] == 0).all() and (o[7] == 0).all()


def test_step_many_rows_of_one_slot():
    """A hundred rows of the batch name one slot, among others: they are its tokens in order."""
    import cfc_recurrent_cell_amd as C
    slots = [(b % 3 != 0) * 1 + (b % 7 == 0) * 2 for b in range(150)]
    c, args, states, sl = step_case(42, "fp32", 150, 5, 1, 2, 48, 36, slots)
    s = torch.from_numpy(states).cuda()
    o = C.delta_rule_step(*args, s, slots=sl)
    for at in range(5):
        mine = [b for b, y in enumerate(slots) if y == at]
        want, fin, _ = R.forward(*(c.x[n][mine] for n in ("q", "k", "v", "g", "beta")),
                                 states[at:at + 1].astype(np.float64), c.scale, [(0, len(mine))])
        c.near(o[mine], want, "o")
        c.near(s[at:at + 1], fin, "states")


def test_steps_are_a_sequence():
    """A prompt, then single tokens: the whole sequence's outputs."""
    import cfc_recurrent_cell_amd as C
    c = Case(43, "bf16", batch=2, length=84, hk=1, hv=2, dk=128, dv=128)
    q, k, v, g, beta = c.args()
    cut = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    o, s = C.delta_rule_forward(*(cut(t, 0, 80) for t in c.args()), initial_state=c.d["s0"])
    outs = [o]
    for t in range(80, 84):
        outs.append(C.delta_rule_step(*(cut(x, t, t + 1)[:, 0] for x in c.args()), s)[:, None])
    c.check_forward(torch.cat(outs, 1), s)


# --------------------------------------------------- streams, graphs, repetition
def test_equal_inputs_give_equal_bits():
    c = Case(51, "bf16", lens=[300, 1, 77], hk=2, hv=4, dk=128, dv=128)
    a = (*c.forward(), *c.backward())
    for _ in range(3):
        for x, y in zip(a, (*c.forward(), *c.backward())):
            assert torch.equal(x, y)


def test_a_sequence_does_not_see_the_others():
    """Values that are not finite stay in their sequence; the chunk they are in and later ones are theirs."""
    a = Case(52, "bf16", lens=[100, 70, 33], hk=1, hv=2, dk=64, dv=64)
    want = (*a.forward(), *a.backward())
    a.d["v"][130] = float("nan")
    a.d["k"][140] = float("inf")
    got = (*a.forward(), *a.backward())
    for i, (x, y) in enumerate(zip(got, want)):
        seq = x.shape[0] == 3
        for part in ([slice(0, 1), slice(2, 3)] if seq else [slice(0, 100), slice(170, 203)]):
            assert torch.equal(x[part], y[part]), i


def test_side_stream_and_given_workspace():
    import cfc_recurrent_cell_amd as C
    c = Case(53, "bf16", batch=2, length=130, hk=1, hv=2, dk=64, dv=64)
    want = (*c.forward(), *c.backward())
    ws = torch.empty(C.delta_rule_workspace(*c.args(), backward=True) + 64, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*c.forward(stream=side, workspace=ws), *c.backward(stream=side, workspace=ws))
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_captured_and_replayed():
    import cfc_recurrent_cell_amd as C
    c = Case(54, "bf16", lens=[130, 5], hk=1, hv=2, dk=64, dv=64)
    step, args, states, sl = step_case(55, "bf16", 3, 4, 1, 2, 64, 64, [2, -1, 2])
    s = torch.from_numpy(states).cuda()
    c.forward(), c.backward(), C.delta_rule_step(*args, s, slots=sl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = (*c.forward(), *c.backward(), C.delta_rule_step(*args, s, slots=sl), s)
    for seed in range(3):
        r = np.random.default_rng(seed)
        for t in (c.d["q"], c.d["v"], args[2]):
            t.copy_(torch.from_numpy(r.standard_normal(t.shape)))
        s.copy_(torch.from_numpy(states))
        for t in out[:-1]:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        s.copy_(torch.from_numpy(states))
        want = (*c.forward(), *c.backward(), C.delta_rule_step(*args, s, slots=sl), s)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_offsets_past_32_bits():
    """Rows 16 MB apart (5 GB of them) and a pool of 9 GB give the bits that small ones give."""
    import cfc_recurrent_cell_amd as C
    n, step = 300, 1 << 23
    c = Case(61, "bf16", batch=1, length=n, hk=1, hv=1, dk=128, dv=128)
    wide = torch.empty(n, step, dtype=torch.bfloat16, device="cuda")
    far = {}
    for i, name in enumerate(("q", "k", "v", "go")):
        far[name] = wide[:, 128 * i:128 * (i + 1)].view(1, n, 1, 128)
        far[name].copy_(c.d[name])
    want = (*c.forward(), *c.backward())
    c.d.update(far)
    for x, y in zip((*c.forward(), *c.backward()), want):
        assert torch.equal(x, y)
    del wide, far
    c = Case(62, "bf16", batch=3, length=1, hk=1, hv=2, dk=128, dv=128)
    args = [c.d[m][:, 0].contiguous() for m in ("q", "k", "v", "g", "beta")]
    pool, slots = 70000, torch.tensor([69999, 4, 40000], dtype=torch.int32, device="cuda")
    states = torch.empty(pool, 2, 128, 128, device="cuda")
    few = c.d["s0"].clone()
    states[slots.long()] = few
    o = C.delta_rule_step(*args, states, slots)
    assert torch.equal(o, C.delta_rule_step(*args, few))
    assert torch.equal(states[slots.long()], few)


def test_two_calls_at_once():
    """Calls on two streams, a workspace each, while both run."""
    a = Case(63, "bf16", batch=2, length=900, hk=2, hv=4, dk=128, dv=128)
    b = Case(64, "bf16", lens=[700, 3, 250], hk=1, hv=2, dk=128, dv=64)
    want = [(*c.forward(), *c.backward()) for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [None, None]
        for i, c in enumerate((a, b)):
            got[i] = (*c.forward(stream=streams[i]), *c.backward(stream=streams[i]))
        torch.cuda.synchronize()
        for x, y in zip(sum(got, ()), sum(want, ())):
            assert torch.equal(x, y)
