"""The kernels that larger calls of the scan, the convolution, the layer norm and the clipping
take: many workgroups, several times 16 channels a workgroup, several sequences a workgroup,
states past the cache, rows wider than 8192, and offsets past 32 bits.  References and
tolerances are those of test_gpu_selective_scan.py, test_gpu_short_conv.py and
test_gpu_layer_norm.py."""
import numpy as np
import pytest

import sequence_reference as R
import test_gpu_layer_norm as L
import test_gpu_selective_scan as S
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


# (16 channels, sequences): beyond 256 pairs the forward has 8 waves instead of 16, from 512 and 1024 on the
# gradients 2 and 4 times 16 channels a workgroup (the last workgroup of a group fewer), and beyond 1024
# workgroups each several sequences
CASES = [("bf16", 130, 1, 16, 60), ("fp32", 130, 1, 16, 120), ("fp16", 90, 2, 7, 100), ("fp32", 33, 3, 3, 180),
         ("bf16", 40, 1, 30, 300), ("fp32", 20, 1, 60, 300), ("fp16", 16, 1, 16, 4200), ("bf16", 528, 1, 2, 64)]


@pytest.mark.parametrize("kind,channels,groups,state,count", CASES)
def test_scan_of_many_sequences(gpu, kind, channels, groups, state, count):
    say(f"[scan] many {kind} {channels} {groups} {state} {count}")
    channels *= groups
    gen = np.random.default_rng(count)
    lens = gen.integers(0, 3 if count > 1000 else 12, count)
    lens[:2] = 70, 9
    rows, tokens, _, offsets = S.layout(list(lens))
    _, p, on = S.inputs(count, kind, tokens, count, channels, groups, state)
    gy, on["gy"] = S.some(gen, S.TYPES[kind], (tokens, channels))
    gf, gfinal = S.some(gen, torch.float32, (count, channels, state))
    args = (on["x"], on["dt"], on["a"], on["b"], on["c"])
    more = dict(d=on["d"], z=on["z"], dt_bias=on["dt_bias"], initial_state=on["initial"], offsets=offsets)
    y, final = gpu.selective_scan_forward(*args, **more)
    got = gpu.selective_scan_backward(*args, on["gy"], grad_final_state=gfinal, **more)
    want, wf, wg = R.scan(p, rows, True, gy, gf)
    size, sf, sg = R.scan(p, rows, True, gy, gf, size=True)
    ulps = S.roundings(p, rows, True)
    S.near(("y", y.dtype), y, want, size, ulps)
    S.near(("final", final.dtype), final, wf, sf, ulps)
    for n, t in zip(R.NAMES, got):
        S.near((n, t.dtype), t, wg[n], sg[n], ulps)


@pytest.mark.parametrize("kind,channels,groups,state,batch", [("bf16", 2064, 1, 16, 70), ("fp32", 2064, 1, 16, 256), ("fp16", 1032, 2, 30, 140),
                                                              ("bf16", 2064, 1, 64, 66), ("fp32", 700, 3, 5, 190), ("fp16", 4100, 1, 3, 40)])
def test_scan_step_of_many_states(gpu, kind, channels, groups, state, batch):
    """From 8192 times 16 channels on a wave has several, and from 32 MB on states pass the cache."""
    say(f"[scan] step of many {kind} {channels} {groups} {state} {batch}")
    channels *= groups
    gen, p, on = S.inputs(batch, kind, batch, batch + 3, channels, groups, state)
    slots = gen.permutation(batch + 3)[:batch]
    slots[3], slots[5], slots[7] = -1, slots[6], slots[6]
    held = on["initial"].clone()
    y = gpu.selective_scan_step(on["x"], on["dt"], on["a"], on["b"], on["c"], held, torch.tensor(slots, dtype=torch.int32).cuda(),
                                d=on["d"], z=on["z"], dt_bias=on["dt_bias"])
    states, sizes = p["initial"].copy(), np.abs(p["initial"])
    pre = np.abs(p["dt"] + p["dt_bias"]).max()
    off = 3 * (64 + 8 + 10 + pre) * 2.0 ** -24  # three tokens of a slot at most
    for b, s in enumerate(slots):
        if s < 0:
            assert (y[b] == 0).all()
            continue
        q = {n: v[b:b + 1] if n in S.ROWS else v for n, v in p.items()}
        size, sizes[s] = (v[0] for v in R.scan({**q, "initial": sizes[s:s + 1]}, R.spans([1]), size=True)[:2])
        want, states[s] = (v[0] for v in R.scan({**q, "initial": states[s:s + 1]}, R.spans([1]))[:2])
        S.near(("y", y.dtype), y[b], want, size, off)
    S.near(("states", torch.float32), held, states, sizes, off)


@pytest.mark.parametrize("kind,channels,width,lens", [("bf16", 2100, 4, [4000, 0, 4, 4100, 30]), ("fp32", 2304, 3, [8192]),
                                                      ("fp16", 9, 2, [1] * 5000 + [0] * 300 + [40])])
def test_conv_of_many_tokens(gpu, kind, channels, width, lens):
    say(f"[conv] many {kind} {channels} {width}")
    rows, tokens, count, offsets = V.layout(lens)
    p, on = V.make(channels, kind, tokens, count, channels, width)
    args = (p["x"], p["w"], p["b"], p["s"], rows, True, p["gy"], p["gf"])
    want, wf, wg = R.conv(*args)
    size, _, sg = R.conv(*args, size=True)
    more = dict(bias=on["b"], initial_state=on["s"], offsets=offsets)
    y, final = gpu.short_conv_forward(on["x"], on["w"], **more)
    V.near("y", y, want, size, 16)
    np.testing.assert_array_equal(final.double().cpu().numpy(), wf)
    got = gpu.short_conv_backward(on["x"], on["w"], on["gy"], grad_final_state=on["gf"], **more)
    for n, t, ulps in zip(("x", "weight", "bias", "initial"), got, (width + 33, 97, 97, width + 33)):
        V.near(n, t, wg[n], sg[n], ulps)


@pytest.mark.parametrize("kind,rows,width", [("bf16", 900, 8200), ("fp32", 9000, 8196), ("fp16", 40, 16383)])
def test_layer_norm_gradients_of_wide_rows(gpu, kind, rows, width):
    """Beyond 8192 columns the weights' terms are summed in 32 bits over 16 rows: 16 roundings more."""
    say(f"[layer norm] wide {kind} {rows} {width}")
    x, w, b, r = L.make(rows, kind, rows, width, "same")
    gy = torch.randn_like(x)
    _, h, mean, rstd = gpu.layer_norm_forward(x, w, b, L.EPS, residual=r)
    gx, gw, gb = gpu.layer_norm_backward(gy, h, w, mean, rstd)
    sums, mags = [torch.zeros(2, width, dtype=torch.float64, device="cuda") for _ in range(2)]
    for at in range(0, rows, 1000):
        part = slice(at, at + 1000)
        rs = rstd[part].double()[:, None]
        n = (h[part].double() - mean[part].double()[:, None]) * rs
        g = gy[part].double()
        d = g * w.double()
        want = rs * (d - d.mean(-1, keepdim=True) - n * (d * n).mean(-1, keepdim=True))
        size = rs * (d.abs() + d.abs().mean(-1, keepdim=True) + n.abs() * (d * n).abs().mean(-1, keepdim=True))
        L.near("x", gx[part], want, size, 64)
        sums += torch.stack([(g * n).sum(0), g.sum(0)])
        mags += torch.stack([(g * n).abs().sum(0), g.abs().sum(0)])
    L.near("weight", gw, sums[0], mags[0], 24)
    L.near("bias", gb, sums[1], mags[1], 24)


def test_offsets_past_32_bits(gpu):
    """Rows, states and elements from 2^31 on, compared with the same ones by themselves."""
    t = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    ch, state, count, length = 4096, 4, 9, 60000
    x = torch.zeros(count, length, ch, dtype=t, device="cuda")  # 2.2e9 elements
    x[-1, :90], x[-1, -90:] = n(90, ch).to(t), n(90, ch).to(t)
    a, bc, w = -torch.exp(n(ch, state)), n(1, length, 1, state).to(t).expand(count, -1, -1, -1).contiguous(), n(ch, 4).to(t)
    say("[scan] 2^31 elements")
    y, final = gpu.selective_scan_forward(x, x, a, bc, bc, z=x)
    one, last = gpu.selective_scan_forward(x[-1:].contiguous(), x[-1:].contiguous(), a, bc[-1:], bc[-1:], z=x[-1:].contiguous())
    # (other blocks of tokens: the same sums in another order)
    assert ((y[-1].float() - one[0].float()).abs() <= 2.0 ** -7 * one[0].float().abs() + 1e-4).all()
    assert ((final[-1] - last[0]).abs() <= 1e-4 * (1 + last[0].abs())).all()
    assert float(one.float().abs().max()) > 1 and (y[:-1] == 0).all()
    del y, one
    say("[conv] 2^31 elements")
    y, final = gpu.short_conv_forward(x, w)
    one, last = gpu.short_conv_forward(x[-1:].contiguous(), w)
    assert torch.equal(y[-1], one[0]) and torch.equal(final[-1], last[0])
    del y, one
    say("[scan] gradients of 2^31 elements")
    got = gpu.selective_scan_backward(x, x, a, bc, bc, x, z=x)
    part = x[-1:].clone()  # (not a view: the clipping changes x)
    want = gpu.selective_scan_backward(part, part, a, bc[-1:], bc[-1:], part, z=part)
    for u, v in zip((got[i] for i in (0, 1, 3, 4, 6)), (want[i] for i in (0, 1, 3, 4, 6))):
        top = float(v.float().abs().max())
        assert top > 0 and ((u[-1].float() - v[0].float()).abs() <= 2.0 ** -7 * v[0].float().abs() + 2e-4 * top).all()
    del got
    say("[conv] gradients of 2^31 elements")
    got = gpu.short_conv_backward(x, w, x)
    want = gpu.short_conv_backward(part, w, part)
    assert torch.equal(got[0][-1], want[0][0])
    assert ((got[1] - want[1]).abs() <= 1e-4 * (1 + want[1].abs())).all()
    del got
    say("[layer norm] 2^31 elements")
    flat, ones = x.view(-1, ch), torch.ones(ch, dtype=t, device="cuda")
    y, h, mean, rstd = gpu.layer_norm_forward(flat, ones, None, 1e-5)
    assert torch.equal(y[-90:], gpu.layer_norm_forward(flat[-90:].contiguous(), ones, None, 1e-5)[0])
    gx, gw, _ = gpu.layer_norm_backward(flat, h, ones, mean, rstd)
    alone = gpu.layer_norm_backward(flat[-90:].contiguous(), h[-90:].contiguous(), ones, mean[-90:].contiguous(), rstd[-90:].contiguous())
    assert torch.equal(gx[-90:], alone[0])
    del y, gx
    say("[clip] 2^31 elements")
    whole = float(part.double().square().sum().sqrt())
    norm = gpu.clip_grad_norm([flat], 0.5 * whole)
    assert abs(float(norm) - whole) <= 2.0 ** -23 * whole
    assert ((x[-1].float() - 0.5 * part[0].float()).abs() <= 2.0 ** -8 * part[0].float().abs()).all()
    del flat, h
    say("[step] pools past 2^31 elements")
    pool = torch.zeros(2 ** 17 + 3, ch, state, device="cuda")
    pool[-2:] = n(2, ch, state)
    few = pool[-2:].clone()
    slots = torch.tensor([2 ** 17 + 1, 2 ** 17 + 2], dtype=torch.int32, device="cuda")
    row, b = n(2, ch).to(t), n(2, 1, state).to(t)
    y = gpu.selective_scan_step(row, row, a, b, b, pool, slots)
    assert torch.equal(y, gpu.selective_scan_step(row, row, a, b, b, few)) and torch.equal(pool[-2:], few)
    assert (pool[:-3] == 0).all()
    del pool
    pool = torch.zeros(2 ** 18, 3, ch, device="cuda", dtype=t)
    pool[-1] = n(3, ch).to(t)
    few = pool[-1:].clone()
    y = gpu.short_conv_step(row[:1], w, pool, torch.tensor([2 ** 18 - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(y, gpu.short_conv_step(row[:1], w, few)) and torch.equal(pool[-1:], few)


def test_long_strides_of_single_tokens(gpu):
    """One token of each row of a long tensor, whose rows are far apart."""
    t, ch, state = torch.float32, 24, 16
    gen = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    far = torch.empty(3, 1 << 21, ch, device="cuda", dtype=t)
    far[:, 7:8] = n(3, 1, ch)
    x = far[:, 7:8]
    a, b, w, s0 = -torch.exp(n(ch, state)), n(3, 1, 1, state), n(ch, 4), n(3, ch, state)
    dense = x.contiguous()
    for u, v in zip(gpu.selective_scan_forward(x, x, a, b, b, z=x, initial_state=s0),
                    gpu.selective_scan_forward(dense, dense, a, b, b, z=dense, initial_state=s0)):
        assert torch.equal(u, v)
    for u, v in zip(gpu.selective_scan_backward(x, x, a, b, b, x, z=x, initial_state=s0),
                    gpu.selective_scan_backward(dense, dense, a, b, b, dense, z=dense, initial_state=s0)):
        assert u is v is None or torch.equal(u, v)
    for u, v in zip((*gpu.short_conv_forward(x, w), *gpu.short_conv_backward(x, w, x)),
                    (*gpu.short_conv_forward(dense, w), *gpu.short_conv_backward(dense, w, dense))):
        assert u is v is None or torch.equal(u, v)


def test_broadcast_rows_with_infinities_are_their_copies(gpu):
    """Rows read at a stride of nothing lie behind the sequence's end too; what is infinite in
    them must not come back from there (0 * inf)."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    ch, state, length = 20, 16, 37
    a, row, bc, z, gy = -torch.exp(n(ch, state)), n(1, 1, ch), n(1, 1, 1, state).abs(), n(1, 1, ch), n(1, 1, ch)
    dt = n(1, length, ch)

    def both(row, bc, z, gy):
        wide = [t.expand(-1, length, *t.shape[2:]) for t in (row, bc, z, gy)]
        out = []
        for x, b, zz, g in (wide, [t.contiguous() for t in wide]):
            out.append((*gpu.selective_scan_forward(x, dt, a, b, b, z=zz),
                        *gpu.selective_scan_backward(x, dt, a, b, b, g, z=zz)))
        for u, v in zip(*out):
            assert (u is v is None) or torch.equal(torch.nan_to_num(u, 7e30), torch.nan_to_num(v, 7e30))
        return out[0]

    inf = lambda t, *at: t.clone().index_put_(tuple(torch.tensor(i, device="cuda") for i in at), torch.tensor(float("inf"), device="cuda"))  # noqa: E731
    both(row, bc, z, gy)
    final = both(inf(row, 0, 0, 3), bc, z, gy)[1]
    assert (final[0, 3] == float("inf")).all() and torch.isfinite(final[0, 4:]).all()
    final = both(row.abs(), inf(bc, 0, 0, 0, 5), z, gy)[1]
    assert (final[0, :, 5] == float("inf")).all() and torch.isfinite(final[0, :, :5]).all()
    both(row, bc, inf(z, 0, 0, 6), gy)
    both(row, bc, z, inf(gy, 0, 0, 7))
