"""Cases and plain forms of the selective scan, the short convolution, the layer norm
and the clipping of gradients.

The selective scan is a recurrent cell whose state h [channels, state] decays by
what the input asks for.  Token t does

    D_t = softplus(dt_t + dt_bias)
    h_t = exp(D_t a) h_{t-1} + D_t x_t b_t^T
    y_t = (h_t c_t + d x_t) silu(z_t)

with a group of channels sharing b_t and c_t.  In front of it a depthwise causal
convolution over the last two to four tokens mixes neighbours:

    y_t = silu(bias + sum_j weight[:, j] x_{t - width + 1 + j})

Both are measured over sequences (all of one length, or packed one behind the other), in
their gradients, and for one token of each sequence of a serving batch with the
states in a pool.

The layer norm's rows are h = x + residual (rounded to the residual stream's type),
y = (h - mean) rstd weight + bias.  Gradients of many tensors are clipped to a
norm over all of them: out = g min(1, max_norm / (norm + 1e-6)).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5
MAX_NORM = 1.0


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a serving batch out of a pool of states, some rows of the batch empty
        {"name": "scan step 256 of a pool of 320", "op": "scan_step", "type": "bf16", "batch": 256, "pool": 320,
         "channels": 4096, "groups": 1, "state": 16, "idle": 13, "gated": True},
        # one long prompt; x and z are halves of one projection, b and c slices of another
        {"name": "scan forward 8192", "op": "scan_forward", "type": "bf16", "lengths": "8192", "packed": False,
         "fused": True, "initial": False, "channels": 4096, "groups": 1, "state": 16, "gated": True},
        # prompts of a serving batch, packed: lengths from nothing to 1500
        {"name": "scan forward packed 16 prompts", "op": "scan_forward", "type": "fp16",
         "lengths": "1500,1,64,700,0,63,65,333,128,1024,2,511,90,257,1200,31", "packed": True, "fused": False,
         "initial": True, "channels": 1536, "groups": 1, "state": 16, "gated": True},
        # a training step's micro-batch
        {"name": "scan backward 4 x 2048", "op": "scan_backward", "type": "bf16", "lengths": "2048*4", "packed": False,
         "fused": False, "initial": False, "channels": 2048, "groups": 1, "state": 16, "gated": True},
        # documents packed for training, sizes that are no powers of two, two groups, no gate
        {"name": "scan backward packed 9 odd fp32", "op": "scan_backward", "type": "fp32",
         "lengths": "77,1000,1,640,333,64,0,129,812", "packed": True, "fused": True, "initial": True,
         "channels": 330, "groups": 2, "state": 12, "gated": False},
        # one conversation: each new token waits for the one before, so this is latency
        {"name": "conv step 1 x 4096", "op": "conv_step", "type": "bf16", "batch": 1, "pool": 1, "channels": 4096,
         "width": 4, "idle": 0, "bias": True, "silu": True},
        # the delta rule's queries, keys and values of a serving batch's prompts: 2 x 16 + 32 heads of 128
        {"name": "conv forward packed 16 prompts", "op": "conv_forward", "type": "bf16",
         "lengths": "1500,1,64,700,0,63,65,333,128,1024,2,511,90,257,1200,31", "packed": True, "fused": False,
         "initial": True, "channels": 8192, "width": 4, "bias": False, "silu": True},
        # a training step's micro-batch, in front of the scan
        {"name": "conv backward 4 x 2048", "op": "conv_backward", "type": "bf16", "lengths": "2048*4", "packed": False,
         "fused": False, "initial": False, "channels": 4096, "width": 4, "bias": True, "silu": True},
        # the norm of a prompt or a training step, the residual stream in 32 bits
        {"name": "layer norm 16384 x 4096", "op": "layer_norm", "type": "bf16", "rows": 16384, "width": 4096,
         "residual": "fp32"},
        # its gradients, a width that is no power of two and an odd row count
        {"name": "layer norm backward 9999 x 1500", "op": "layer_norm_backward", "type": "bf16", "rows": 9999,
         "width": 1500, "stream": True},
        # the training-scale CfC cell's gradients: w_in, w_rec, b and w_tau at 128 inputs and 128 units
        {"name": "clip the cell's gradients", "op": "clip", "type": "fp32", "sizes": "16384*2,128*2"},
        # a model's gradients: six layers' matrices and vectors, an odd one and one embedding
        {"name": "clip 62 gradients", "op": "clip", "type": "bf16",
         "sizes": "8388608*18,2097152*18,131072*6,4096*12,2048*6,1001,67108864"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_step", "scan_forward", "scan_forward", "scan_backward", "scan_backward", "conv_step",
                     "conv_forward", "conv_backward", "layer_norm", "layer_norm_backward", "clip"])
    case = {"op": op, "type": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    if op.startswith("layer_norm"):
        rows, width = _log_int(rng, 1, 16384), _log_int(rng, 1, 8192)
        if rng.random() < 0.5:
            width = -(-width // 8) * 8
        while rows * width > 1 << 26:
            rows //= 2
        case.update(rows=rows, width=width)
        if op == "layer_norm":
            case["residual"] = rng.choice(["none", "same", "fp32"])
        else:
            case["stream"] = rng.random() < 0.5
        return case
    if op == "clip":
        parts, room, left = [], 1 << 26, 60
        for _ in range(_log_int(rng, 1, 12)):
            n = _log_int(rng, 1, 1 << 22)
            count = max(1, min(_log_int(rng, 1, 40), room // n, left - 12))
            room, left = max(0, room - n * count), left - count
            parts.append("%d*%d" % (n, count))
        case["sizes"] = ",".join(parts)
        return case
    if op.startswith("scan"):
        groups = rng.choice([1, 1, 1, 2, 3])
        case.update(channels=groups * _log_int(rng, 1, 2048 // groups), groups=groups,
                    state=rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 64)]), gated=rng.random() < 0.7)
        size = case["channels"] * case["state"]
    else:
        case.update(channels=_log_int(rng, 1, 8192), width=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5,
                    silu=rng.random() < 0.7)
        if rng.random() < 0.5:
            case["channels"] = -(-case["channels"] // 8) * 8
        size = case["channels"] * 8
    if op.endswith("step"):
        batch = _log_int(rng, 1, 256)
        case.update(batch=batch, pool=batch + rng.randint(0, 64), idle=rng.randint(0, batch // 4))
        return case
    # so many tokens that a draw costs no more than the listed cases
    room = max(1, min(16384, (1 << 27 if op.endswith("backward") else 1 << 28) // size))
    count = _log_int(rng, 1, 24)
    if rng.random() < 0.5:
        length = _log_int(rng, 1, min(room, 4096))
        case.update(lengths="%d*%d" % (length, max(1, min(count, room // length))), packed=False)
    else:
        lengths = []
        for _ in range(count):
            n = 0 if rng.random() < 0.1 else _log_int(rng, 1, 1500)
            n = min(n, room)
            room -= n
            lengths.append(n)
        lengths[0] = max(1, lengths[0])
        case.update(lengths=",".join(map(str, lengths)), packed=True)
    case.update(fused=rng.random() < 0.4, initial=rng.random() < 0.5)
    return case


def _numbers(text):
    out = []
    for part in text.split(","):
        n, _, count = part.partition("*")
        out += [int(n)] * int(count or 1)
    return out


# ------------------------------------------------------------------- the inputs
def prepare(case, seed):
    dev, op = "cuda", case["op"]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev, dtype=torch.float32)

    def slots_of():
        if case["pool"] == 1:
            return None
        slots = torch.randperm(case["pool"], generator=gen, device=dev)[:case["batch"]].to(torch.int32)
        if case["idle"]:
            slots[torch.randperm(case["batch"], generator=gen, device=dev)[:case["idle"]]] = -1
        return slots

    s = {"case": case}
    if op.startswith("layer_norm"):
        rows, width = case["rows"], case["width"]
        s["weight"] = (1 + 0.2 * normal(width)).to(dtype)
        if op == "layer_norm_backward":
            h = (1.5 * normal(rows, width) + 0.5 * normal(rows, 1)).to(dtype)
            s["h"], wide = h, h.float()
            s["mean"] = wide.mean(-1)
            s["rstd"] = torch.rsqrt((wide - s["mean"][:, None]).square().mean(-1) + EPS)
            s["grad_y"] = normal(rows, width).to(dtype)
            s["grad_h"] = normal(rows, width).to(dtype) if case["stream"] else None
        else:
            s["bias"] = (0.2 * normal(width)).to(dtype)
            s["x"] = normal(rows, width).to(dtype)
            kind = case["residual"]
            s["residual"] = None
            if kind != "none":
                s["residual"] = (normal(rows, width) + 0.5 * normal(rows, 1)).to(dtype if kind == "same" else torch.float32)
        return s

    if op == "clip":
        # gradients of a few thousandths, another size for each tensor; the clipped ones go to buffers of their own
        s["grads"] = [(normal(n) * 10 ** -(2 + 2 * float(i % 7) / 6)).to(dtype) for i, n in enumerate(_numbers(case["sizes"]))]
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
        return s

    ch = case["channels"]
    if op.startswith("scan"):
        groups, n = case["groups"], case["state"]
        # decays: a from -1 to -state and rates from a thousandth to a tenth, as such layers begin
        s["a"] = -(torch.arange(1, n + 1, device=dev) * torch.exp(0.1 * normal(ch, n)))
        rate = torch.exp(math.log(1e-3) + uniform(ch) * math.log(100.0))
        s["dt_bias"] = rate + torch.log(-torch.expm1(-rate))
        s["d"] = 1 + 0.1 * normal(ch)
        if op == "scan_step":
            b = case["batch"]
            s.update(x=normal(b, ch).to(dtype), dt=normal(b, ch).to(dtype), b=normal(b, groups, n).to(dtype),
                     c=normal(b, groups, n).to(dtype), z=normal(b, ch).to(dtype) if case["gated"] else None,
                     pool=0.3 * normal(case["pool"], ch, n), slots=slots_of())
            return s
    else:
        s["weight"] = (case["width"] ** -0.5 * normal(ch, case["width"])).to(dtype)
        s["bias"] = (0.1 * normal(ch)).to(dtype) if case["bias"] else None
        if op == "conv_step":
            s.update(x=normal(case["batch"], ch).to(dtype), pool=normal(case["pool"], case["width"] - 1, ch).to(dtype),
                     slots=slots_of())
            return s

    lens = _numbers(case["lengths"])
    lead = (sum(lens),) if case["packed"] else (len(lens), lens[0])
    s["lens"], s["offsets"] = lens, None
    if case["packed"]:
        ends = [0]
        for length in lens:
            ends.append(ends[-1] + length)
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=dev)
    if op.startswith("scan"):
        width = groups * n
        if case["fused"]:
            # slices of the projections' outputs, where they lie
            row = normal(*lead, 2 * ch).to(dtype)
            s["x"], s["z"] = row[..., :ch], row[..., ch:]
            low = normal(*lead, 8 + 2 * width).to(dtype)
            s["b"] = low[..., 8:8 + width].unflatten(-1, (groups, n))
            s["c"] = low[..., 8 + width:].unflatten(-1, (groups, n))
        else:
            s["x"], s["z"] = normal(*lead, ch).to(dtype), normal(*lead, ch).to(dtype)
            s["b"], s["c"] = (normal(*lead, groups, n).to(dtype) for _ in range(2))
        if not case["gated"]:
            s["z"] = None
        s["dt"] = normal(*lead, ch).to(dtype)
        s["initial"] = 0.3 * normal(len(lens), ch, n) if case["initial"] else None
        if op == "scan_backward":
            s["grad_final"] = 0.1 * normal(len(lens), ch, n) if case["initial"] else None
    else:
        s["x"] = normal(*lead, ch + 24).to(dtype)[..., 8:8 + ch] if case["fused"] else normal(*lead, ch).to(dtype)
        s["initial"] = normal(len(lens), case["width"] - 1, ch).to(dtype) if case["initial"] else None
        if op == "conv_backward":
            s["grad_final"] = normal(len(lens), case["width"] - 1, ch).to(dtype) if case["initial"] else None
    if op.endswith("backward"):
        s["grad_y"] = normal(*lead, ch).to(dtype)
    return s


# -------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(op, s)
    plain = {"scan_step": _plain_scan_step, "scan_forward": _plain_scan_forward, "scan_backward": _plain_scan_backward,
             "conv_step": _plain_conv_step, "conv_forward": _plain_conv_forward, "conv_backward": _plain_conv_backward,
             "layer_norm": _plain_norm, "layer_norm_backward": _plain_norm_backward, "clip": _plain_clip}
    return plain[op](s)


def _run_own(op, s):
    import cfc_recurrent_cell_amd as cfc
    if op == "scan_step":
        y = cfc.selective_scan_step(s["x"], s["dt"], s["a"], s["b"], s["c"], s["pool"], slots=s["slots"], d=s["d"],
                                    z=s["z"], dt_bias=s["dt_bias"])
        return {"y": y, "pool": s["pool"]}
    if op == "scan_forward":
        y, final = cfc.selective_scan_forward(s["x"], s["dt"], s["a"], s["b"], s["c"], d=s["d"], z=s["z"],
                                              dt_bias=s["dt_bias"], initial_state=s["initial"], offsets=s["offsets"])
        return {"y": y, "final": final}
    if op == "scan_backward":
        names = ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "initial")
        grads = cfc.selective_scan_backward(s["x"], s["dt"], s["a"], s["b"], s["c"], s["grad_y"], d=s["d"], z=s["z"],
                                            dt_bias=s["dt_bias"], initial_state=s["initial"],
                                            grad_final_state=s["grad_final"], offsets=s["offsets"])
        return dict(zip(names, grads))
    if op.startswith("conv"):
        act = "silu" if s["case"]["silu"] else None
        if op == "conv_step":
            y = cfc.short_conv_step(s["x"], s["weight"], s["pool"], slots=s["slots"], bias=s["bias"], activation=act)
            return {"y": y, "pool": s["pool"]}
        if op == "conv_forward":
            y, final = cfc.short_conv_forward(s["x"], s["weight"], bias=s["bias"], initial_state=s["initial"],
                                              activation=act, offsets=s["offsets"])
            return {"y": y, "final": final}
        grads = cfc.short_conv_backward(s["x"], s["weight"], s["grad_y"], bias=s["bias"], initial_state=s["initial"],
                                        grad_final_state=s["grad_final"], activation=act, offsets=s["offsets"])
        return dict(zip(("x", "weight", "bias", "initial"), grads))
    if op == "layer_norm":
        y, h, mean, rstd = cfc.layer_norm_forward(s["x"], s["weight"], s["bias"], EPS, residual=s["residual"])
        return {"y": y, "h": h, "mean": mean, "rstd": rstd}
    if op == "layer_norm_backward":
        gx, gw, gb = cfc.layer_norm_backward(s["grad_y"], s["h"], s["weight"], s["mean"], s["rstd"], grad_h=s["grad_h"])
        return {"x": gx, "weight": gw, "bias": gb}
    norm = cfc.clip_grad_norm(s["grads"], MAX_NORM, out=s["out"])
    return {"norm": norm, "out": s["out"]}


# ---------------------------------------------------- plain forms in 32 bits
def _plain_norm(s):
    x, w = s["x"].float(), s["weight"].float()
    h = s["x"] if s["residual"] is None else (x + s["residual"].float()).to(s["residual"].dtype)
    hf = h.float()
    mean = hf.mean(-1, keepdim=True)
    rstd = torch.rsqrt((hf - mean).square().mean(-1, keepdim=True) + EPS)
    y = (hf - mean) * rstd * w + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "h": h, "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_backward(s):
    h, w, dy = s["h"].float(), s["weight"].float(), s["grad_y"].float()
    rstd = s["rstd"][:, None]
    n = (h - s["mean"][:, None]) * rstd
    dn = dy * w
    gx = rstd * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
    if s["grad_h"] is not None:
        gx = gx + s["grad_h"].float()
    return {"x": gx.to(s["h"].dtype), "weight": (dy * n).sum(0, dtype=torch.float64).float(),
            "bias": dy.sum(0, dtype=torch.float64).float()}


def _plain_clip(s):
    total = torch.stack([g.double().square().sum() for g in s["grads"]]).sum()
    norm = total.sqrt().float()
    factor = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": norm, "out": [(g.float() * factor).to(g.dtype) for g in s["grads"]]}


def _softplus(t):
    return t.clamp_min(0) + torch.log1p(torch.exp(-t.abs()))


def _rows(s, name):
    """Input `name` in 32 bits with one axis of all sequences' tokens."""
    t = s[name]
    return t.flatten(0, 0 if s["case"]["packed"] else 1).float()


def _ends(s):
    """The first and the last row of each sequence that has any, and which sequences those are."""
    lens = torch.tensor(s["lens"], device=s["x"].device)
    ends = lens.cumsum(0)
    some = torch.nonzero(lens > 0)[:, 0]
    return (ends - lens)[some], ends[some] - 1, some


def _scan(decay, add, longest):
    """h_t = decay_t h_{t-1} + add_t along the first axis, by doubling; a decay of zero begins anew."""
    step = 1
    while step < longest:
        add = torch.cat([add[:step], add[step:] + decay[step:] * add[:-step]])
        decay = torch.cat([decay[:step], decay[step:] * decay[:-step]])
        step *= 2
    return add


def _scan_inputs(s):
    case = s["case"]
    share = case["channels"] // case["groups"]
    x, pre = _rows(s, "x"), _rows(s, "dt") + s["dt_bias"]
    b, c = (_rows(s, n).repeat_interleave(share, 1) for n in ("b", "c"))
    step = _softplus(pre)
    decay = torch.exp(step[..., None] * s["a"])
    add = (step * x)[..., None] * b
    first, last, some = _ends(s)
    kept = decay[first]
    if s["initial"] is not None:
        add[first] += kept * s["initial"][some]
    return x, pre, b, c, step, decay, add, first, last, some


def _states(decay, add, first, longest):
    decay = decay.clone()
    decay[first] = 0
    return _scan(decay, add, longest)


def _plain_scan_forward(s):
    x, _, b, c, _, decay, add, first, last, some = _scan_inputs(s)
    h = _states(decay, add, first, max(s["lens"]))
    y = (h * c).sum(-1) + s["d"] * x
    if s["z"] is not None:
        z = _rows(s, "z")
        y = y * z * torch.sigmoid(z)
    final = torch.zeros(len(s["lens"]), *s["a"].shape, device=x.device) if s["initial"] is None else s["initial"].clone()
    final[some] = h[last]
    return {"y": y.to(s["x"].dtype).view(s["x"].shape), "final": final}


def _plain_scan_backward(s):
    case, kind = s["case"], s["x"].dtype
    x, pre, b, c, step, decay, add, first, last, some = _scan_inputs(s)
    longest = max(s["lens"])
    h = _states(decay, add, first, longest)
    gy, out = _rows(s, "grad_y"), {}
    grad_z = None
    if s["z"] is not None:
        z = _rows(s, "z")
        sig = torch.sigmoid(z)
        grad_z = gy * ((h * c).sum(-1) + s["d"] * x) * (sig * (1 + z * (1 - sig)))
        gy = gy * z * sig
    # the states' gradients from the last token to the first
    gh = gy[..., None] * c
    if s["grad_final"] is not None:
        gh[last] += s["grad_final"][some]
    after = torch.cat([decay[1:], torch.zeros_like(decay[:1])])
    after[last] = 0
    gh = _scan(after.flip(0), gh.flip(0), longest).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = 0 if s["initial"] is None else s["initial"][some]
    to_decay = gh * decay * before
    gu = (gh * b).sum(-1)
    gstep = gu * x + (to_decay * s["a"]).sum(-1)
    gdt = gstep * torch.sigmoid(pre)
    groups, n = case["groups"], case["state"]
    out["x"] = (gu * step + s["d"] * gy).to(kind).view(s["x"].shape)
    out["dt"] = gdt.to(kind).view(s["x"].shape)
    out["a"] = (to_decay * step[..., None]).sum(0, dtype=torch.float64).float()
    for name, t in (("b", gh * (step * x)[..., None]), ("c", gy[..., None] * h)):
        out[name] = t.view(t.shape[0], groups, -1, n).sum(2).to(kind).view(s[name].shape)
    out["d"] = (gy * x).sum(0, dtype=torch.float64).float()
    out["z"] = None if grad_z is None else grad_z.to(kind).view(s["x"].shape)
    out["dt_bias"] = gdt.sum(0, dtype=torch.float64).float()
    out["initial"] = None
    if s["initial"] is not None:
        out["initial"] = torch.zeros_like(s["initial"]) if s["grad_final"] is None else s["grad_final"].clone()
        out["initial"][some] = decay[first] * gh[first]
    return out


def _plain_scan_step(s):
    case = s["case"]
    share = case["channels"] // case["groups"]
    x = s["x"].float()
    rows = torch.arange(case["batch"], device=x.device)
    at = rows if s["slots"] is None else s["slots"].long()
    rows, at = rows[at >= 0], at[at >= 0]
    b, c = (s[n].float()[rows].repeat_interleave(share, 1) for n in ("b", "c"))
    step = _softplus(s["dt"].float()[rows] + s["dt_bias"])
    h = torch.exp(step[..., None] * s["a"]) * s["pool"][at] + (step * x[rows])[..., None] * b
    s["pool"][at] = h
    got = (h * c).sum(-1) + s["d"] * x[rows]
    if s["z"] is not None:
        z = s["z"].float()[rows]
        got = got * z * torch.sigmoid(z)
    y = torch.zeros_like(x)
    y[rows] = got
    return {"y": y.to(s["x"].dtype), "pool": s["pool"]}


def _taps(s):
    """For each tap the inputs that it meets, and the rows and the kept inputs that they come from."""
    width, x = s["case"]["width"], _rows(s, "x")
    lens = torch.tensor(s["lens"], device=x.device)
    starts = lens.cumsum(0) - lens
    seq = torch.repeat_interleave(torch.arange(len(s["lens"]), device=x.device), lens)
    row = torch.arange(x.shape[0], device=x.device)
    place = row - starts[seq]
    kept = None if s["initial"] is None else s["initial"].float()
    taps = []
    for j in range(width):
        back = width - 1 - j
        inside = place >= back
        t = torch.where(inside[:, None], x[(row - back).clamp_min(0)], torch.zeros_like(x))
        if kept is not None:
            # place p of a sequence meets kept input p + j
            t = torch.where(inside[:, None], t, kept[seq, (place + j).clamp(max=width - 2)])
        taps.append(t)
    return taps, seq, place, row


def _conv_pre(s, taps):
    w = s["weight"].float()
    pre = sum(t * w[:, j] for j, t in enumerate(taps))
    return pre if s["bias"] is None else pre + s["bias"].float()


def _plain_conv_forward(s):
    case, width = s["case"], s["case"]["width"]
    taps, _, _, _ = _taps(s)
    y = _conv_pre(s, taps)
    if case["silu"]:
        y = y * torch.sigmoid(y)
    x = s["x"].flatten(0, 0 if case["packed"] else 1)
    count = len(s["lens"])
    lens = torch.tensor(s["lens"], device=x.device)
    place = lens[:, None] - (width - 1) + torch.arange(width - 1, device=x.device)
    rows = (lens.cumsum(0) - lens)[:, None] + place.clamp_min(0)
    final = x[rows.clamp(max=x.shape[0] - 1)]
    kept = s["initial"] if s["initial"] is not None else torch.zeros(count, width - 1, x.shape[1], device=x.device, dtype=x.dtype)
    old = torch.gather(kept, 1, (place + width - 1).clamp(max=width - 2)[..., None].expand_as(kept))
    final = torch.where((place >= 0)[..., None], final, old)
    return {"y": y.to(x.dtype).view(s["x"].shape), "final": final}


def _plain_conv_backward(s):
    case, width = s["case"], s["case"]["width"]
    taps, seq, place, row = _taps(s)
    gp = _rows(s, "grad_y")
    if case["silu"]:
        pre = _conv_pre(s, taps)
        sig = torch.sigmoid(pre)
        gp = gp * (sig * (1 + pre * (1 - sig)))
    w = s["weight"].float()
    lens = torch.tensor(s["lens"], device=gp.device)
    left = lens[seq] - 1 - place  # tokens of the sequence behind this one
    gx = torch.zeros_like(gp)
    for j in range(width):
        ahead = width - 1 - j
        there = (left >= ahead)[:, None]
        gx += torch.where(there, gp[(row + ahead).clamp(max=gp.shape[0] - 1)], torch.zeros_like(gp)) * w[:, j]
    initial = None
    if s["grad_final"] is not None:
        # the last tokens are kept too
        g = s["grad_final"].float()
        gx += torch.where((left < width - 1)[:, None], g[seq, (width - 2 - left).clamp_min(0)], torch.zeros_like(gx))
    if s["initial"] is not None:
        # a kept input i meets the tokens of places up to i, and is kept on by sequences shorter than the state
        initial = torch.zeros(s["initial"].shape, device=gp.device)
        starts = lens.cumsum(0) - lens
        for i in range(width - 1):
            for p in range(i + 1):
                there = (lens > p)[:, None]
                initial[:, i] += torch.where(there, gp[(starts + p).clamp(max=gp.shape[0] - 1)], torch.zeros_like(initial[:, i])) * w[:, i - p]
            if s["grad_final"] is not None:
                to = i - lens
                initial[:, i] += torch.where((to >= 0)[:, None], g[torch.arange(len(lens), device=g.device), to.clamp_min(0)], torch.zeros_like(initial[:, i]))
        initial = initial.to(s["x"].dtype)
    weight = torch.stack([(gp * t).sum(0, dtype=torch.float64) for t in taps], 1).float()
    bias = None if s["bias"] is None else gp.sum(0, dtype=torch.float64).float()
    return {"x": gx.to(s["x"].dtype).view(s["x"].shape), "weight": weight, "bias": bias, "initial": initial}


def _plain_conv_step(s):
    case = s["case"]
    x = s["x"]
    rows = torch.arange(case["batch"], device=x.device)
    at = rows if s["slots"] is None else s["slots"].long()
    rows, at = rows[at >= 0], at[at >= 0]
    window = torch.cat([s["pool"][at], x[rows][:, None]], 1)
    got = (window.float() * s["weight"].float().t()).sum(1)
    if s["bias"] is not None:
        got = got + s["bias"].float()
    if case["silu"]:
        got = got * torch.sigmoid(got)
    s["pool"][at] = window[:, 1:]
    y = torch.zeros_like(x)
    y[rows] = got.to(x.dtype)
    return {"y": y, "pool": s["pool"]}


# ------------------------------------------- what the definition gives, in 64 bits
def exact(case, seed):
    op, s = case["op"], prepare(case, seed)
    if op.startswith("layer_norm"):
        return _exact_norm(op, s)
    if op == "clip":
        squares = torch.zeros((), dtype=torch.float64, device="cuda")
        for g in s["grads"]:
            squares += torch.linalg.vector_norm(g.double()) ** 2
        norm = squares ** 0.5
        small = min(1.0, MAX_NORM / (float(norm) + 1e-6))
        return {"norm": norm, "out": [g.double() * small for g in s["grads"]]}
    if op.startswith("scan"):
        return _exact_scan_step(case, s) if op == "scan_step" else _exact_scan(case, s)
    return _exact_conv_step(case, s) if op == "conv_step" else _exact_conv(case, s)


def _exact_norm(op, s):
    w = s["weight"].double()
    if op == "layer_norm":
        h = s["x"].double()
        if s["residual"] is not None:  # the stream is kept in its own type, and the norm is that of what is kept
            h = (h + s["residual"].double()).to(s["residual"].dtype).double()
        mean = h.sum(-1) / h.shape[-1]
        away = h - mean[:, None]
        rstd = 1 / torch.sqrt((away * away).sum(-1) / h.shape[-1] + EPS)
        return {"y": away * rstd[:, None] * w + s["bias"].double(), "h": h, "mean": mean, "rstd": rstd}
    dy, rstd = s["grad_y"].double(), s["rstd"].double()[:, None]
    away = s["h"].double() - s["mean"].double()[:, None]
    g, count = dy * w, dy.shape[-1]
    gx = rstd * g - (rstd / count) * g.sum(-1, keepdim=True) - away * (rstd ** 3 / count) * (g * away).sum(-1, keepdim=True)
    if s["grad_h"] is not None:
        gx = gx + s["grad_h"].double()
    return {"x": gx, "weight": (dy * away * rstd).sum(0), "bias": dy.sum(0)}


def _silu(t):
    return t / (1 + torch.exp(-t))


def _silu_slope(t):
    e = torch.exp(-t)
    return 1 / (1 + e) + t * e / (1 + e) ** 2


def _wide_softplus(t):
    return torch.where(t > 0, t + torch.log1p(torch.exp(-t.abs())), torch.log1p(torch.exp(-t.abs())))


def _live(case, s):
    slots = list(range(case["batch"])) if s["slots"] is None else s["slots"].tolist()
    return [(row, at) for row, at in enumerate(slots) if at >= 0]


def _exact_scan_step(case, s):
    share = case["channels"] // case["groups"]
    pool = s["pool"].double()
    y = torch.zeros(case["batch"], case["channels"], dtype=torch.float64, device=pool.device)
    for row, at in _live(case, s):
        b, c = (s[n][row].double().repeat_interleave(share, 0) for n in ("b", "c"))
        x = s["x"][row].double()
        step = _wide_softplus(s["dt"][row].double() + s["dt_bias"].double())
        pool[at] = torch.exp(step[:, None] * s["a"].double()) * pool[at] + (step * x)[:, None] * b
        y[row] = torch.einsum("dn,dn->d", pool[at], c) + s["d"].double() * x
        if s["z"] is not None:
            y[row] *= _silu(s["z"][row].double())
    return {"y": y, "pool": pool}


def _columns(case, lens, t):
    """[..., features] of the sequences as [longest, sequence, features] in 64 bits, zero behind their ends."""
    flat = t.double().reshape(-1, *t.shape[1 if case["packed"] else 2:])
    out = torch.zeros(max(lens), len(lens), *flat.shape[1:], dtype=torch.float64, device=t.device)
    start = 0
    for i, n in enumerate(lens):
        out[:n, i] = flat[start:start + n]
        start += n
    return out


def _back(lens, t, like):
    return torch.cat([t[:n, i] for i, n in enumerate(lens)]).reshape(like.shape)


def _exact_scan(case, s):
    lens, back = s["lens"], case["op"] == "scan_backward"
    longest, count, ch, n = max(lens), len(lens), case["channels"], case["state"]
    if back and longest * count * ch * n * 8 > 80e9:
        return None
    share = ch // case["groups"]
    a, d, bias = s["a"].double(), s["d"].double(), s["dt_bias"].double()
    x, dt, b, c = (_columns(case, lens, s[m]) for m in ("x", "dt", "b", "c"))
    z = None if s["z"] is None else _columns(case, lens, s["z"])
    alive = torch.tensor(lens, device=x.device)[None] > torch.arange(longest, device=x.device)[:, None]
    step = _wide_softplus(dt + bias) * alive[..., None]  # a step of nothing leaves the state as it is
    h = torch.zeros(count, ch, n, dtype=torch.float64, device=x.device)
    if s["initial"] is not None:
        h = s["initial"].double()
    states, pre = [], torch.zeros_like(x)
    for t in range(longest):
        if back:
            states.append(h)
        bt, ct = (m[t].repeat_interleave(share, 1) for m in (b, c))
        h = torch.exp(step[t][..., None] * a) * h + (step[t] * x[t])[..., None] * bt
        pre[t] = torch.einsum("sdn,sdn->sd", h, ct) + d * x[t]
    if not back:
        return {"y": _back(lens, pre if z is None else pre * _silu(z), s["x"]), "final": h}
    gy = _columns(case, lens, s["grad_y"])
    gz = None
    if z is not None:
        gz = gy * pre * _silu_slope(z)
        gy = gy * _silu(z)
    gx, gstep, gb, gc = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(b), torch.zeros_like(c)
    ga = torch.zeros_like(a)
    gh = torch.zeros_like(h) if s["grad_final"] is None else s["grad_final"].double()
    for t in reversed(range(longest)):
        bt, ct = (m[t].repeat_interleave(share, 1) for m in (b, c))
        decay = torch.exp(step[t][..., None] * a)
        after = decay * states[t] + (step[t] * x[t])[..., None] * bt
        gc[t] = (gy[t][..., None] * after).view(count, case["groups"], share, n).sum(2)
        gh = gh + gy[t][..., None] * ct
        into = gh * decay * states[t]
        ga += torch.einsum("sdn,sd->dn", into, step[t])
        gu = torch.einsum("sdn,sdn->sd", gh, bt)
        gb[t] = (gh * (step[t] * x[t])[..., None]).view(count, case["groups"], share, n).sum(2)
        gx[t] = gu * step[t] + d * gy[t]
        gstep[t] = gu * x[t] + torch.einsum("sdn,dn->sd", into, a)
        gh = gh * decay
        states[t] = None
    gdt = gstep * alive[..., None] / (1 + torch.exp(-(dt + bias)))
    out = {m: _back(lens, t, s[m]) for m, t in (("x", gx), ("dt", gdt), ("b", gb), ("c", gc))}
    out.update(a=ga, d=(gy * x).sum((0, 1)), dt_bias=gdt.sum((0, 1)), z=None if gz is None else _back(lens, gz, s["z"]),
               initial=gh if s["initial"] is not None else None)
    return {m: out[m] for m in ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "initial")}


def _exact_conv_step(case, s):
    pool = s["pool"].double()
    y = torch.zeros(case["batch"], case["channels"], dtype=torch.float64, device=pool.device)
    w = s["weight"].double()
    for row, at in _live(case, s):
        seen = torch.cat([pool[at], s["x"][row].double()[None]])
        got = torch.einsum("jd,dj->d", seen, w)
        if s["bias"] is not None:
            got = got + s["bias"].double()
        y[row] = _silu(got) if case["silu"] else got
        pool[at] = seen[1:]
    return {"y": y, "pool": pool}


def _exact_conv(case, s):
    back, width, w = case["op"] == "conv_backward", case["width"], s["weight"].double()
    flat = s["x"].reshape(-1, case["channels"])
    gflat = s["grad_y"].reshape(-1, case["channels"]) if back else None
    ys, finals, gxs, ginit, start = [], [], [], [], 0
    gw = torch.zeros_like(w)
    gbias = torch.zeros(case["channels"], dtype=torch.float64, device=w.device)
    for i, n in enumerate(s["lens"]):
        kept = torch.zeros(width - 1, case["channels"], dtype=torch.float64, device=w.device)
        if s["initial"] is not None:
            kept = s["initial"][i].double()
        seen = torch.cat([kept, flat[start:start + n].double()])
        pre = torch.zeros(n, case["channels"], dtype=torch.float64, device=w.device)
        for j in range(width):
            pre += seen[j:j + n] * w[:, j]
        if s["bias"] is not None:
            pre += s["bias"].double()
        ys.append(_silu(pre) if case["silu"] else pre)
        finals.append(seen[n:])
        if back:
            g = gflat[start:start + n].double()
            if case["silu"]:
                g = g * _silu_slope(pre)
            gseen = torch.zeros_like(seen)
            for j in range(width):
                gseen[j:j + n] += g * w[:, j]
                gw[:, j] += (g * seen[j:j + n]).sum(0)
            if s["grad_final"] is not None:
                gseen[n:] += s["grad_final"][i].double()
            gbias += g.sum(0)
            ginit.append(gseen[:width - 1])
            gxs.append(gseen[width - 1:])
        start += n
    if not back:
        return {"y": torch.cat(ys).view(s["x"].shape), "final": torch.stack(finals)}
    return {"x": torch.cat(gxs).view(s["x"].shape), "weight": gw, "bias": gbias if s["bias"] is not None else None,
            "initial": torch.stack(ginit) if s["initial"] is not None else None}


# --------------------------------------------------------------------- the work
def work(case):
    size, op = BYTES[case["type"]], case["op"]
    if op.startswith("layer_norm"):
        rows, width = case["rows"], case["width"]
        n = rows * width
        if op == "layer_norm_backward":
            return {"bytes": n * size * (4 if case["stream"] else 3) + rows * 8 + width * (size + 8), "flops": 12 * n}
        h = {"none": 0, "same": 2 * size, "fp32": 8}[case["residual"]]
        return {"bytes": n * (2 * size + h) + rows * 8 + 2 * width * size, "flops": 8 * n}
    if op == "clip":
        n = sum(_numbers(case["sizes"]))
        return {"bytes": 2 * n * size + 4, "flops": 3 * n}
    ch = case["channels"]
    if op.startswith("scan"):
        state, shared = ch * case["state"], 2 * case["groups"] * case["state"]
        token = ch * (3 if case["gated"] else 2) + shared  # x, dt, z, b and c
        once = 4 * state + 8 * ch
        if op == "scan_step":
            b = case["batch"] - case["idle"]
            return {"bytes": b * ((token + ch) * size + 8 * state) + once, "flops": 7 * b * state}
        lens = _numbers(case["lengths"])
        tokens, kept = sum(lens), 4 * len(lens) * state
        if op == "scan_forward":
            return {"bytes": tokens * (token + ch) * size + once + kept * (2 if case["initial"] else 1),
                    "flops": 7 * tokens * state}
        return {"bytes": tokens * (2 * token + ch) * size + 2 * once + (3 * kept if case["initial"] else 0),
                "flops": 20 * tokens * state}
    width = case["width"]
    state = (width - 1) * ch * size
    weights = ch * (width + (1 if case["bias"] else 0))
    if op == "conv_step":
        b = case["batch"] - case["idle"]
        return {"bytes": b * (2 * ch * size + 2 * state) + weights * size, "flops": b * ch * 2 * width}
    lens = _numbers(case["lengths"])
    tokens, kept = sum(lens), len(lens) * state
    if op == "conv_forward":
        return {"bytes": 2 * tokens * ch * size + weights * size + kept * (2 if case["initial"] else 1),
                "flops": tokens * ch * 2 * width}
    return {"bytes": 3 * tokens * ch * size + weights * (size + 4) + (3 * kept if case["initial"] else 0),
            "flops": tokens * ch * 6 * width}
