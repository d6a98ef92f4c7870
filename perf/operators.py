"""Cases and plain forms of the gated delta rule and of the root-mean-square norm.

The gated delta rule is a recurrent cell with a matrix state S [dim_k, dim_v]
for each head.  Token t decays the state, corrects what it answers for the key
k_t towards v_t, and reads it with q_t:

    S'  = exp(g_t) S_{t-1}
    u_t = beta_t (v_t - S'^T k_t)
    S_t = S' + k_t u_t^T
    o_t = scale S_t^T q_t

Value head h reads key head h // (heads_v / heads_k).  Three forms of it are
measured: over sequences (all of one length, or packed one behind the other),
its gradients, and one token for each sequence of a serving batch with the
states in a pool.

The norm's rows are h = x + residual (rounded to the residual stream's type),
y = h * rstd * weight with rstd = 1 / sqrt(mean(h^2) + eps); y is also given in
e4m3 with one scale for each row or for each group of columns.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
CHUNK = 64
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one conversation: each new token waits for the one before, so this is latency
        {"name": "step 1 x 32 heads", "op": "step", "type": "bf16", "batch": 1, "pool": 1, "heads_k": 16,
         "heads_v": 32, "dim_k": 128, "dim_v": 128, "idle": 0},
        # a serving batch out of a pool of states, some rows of the batch empty
        {"name": "step 256 of a pool of 320", "op": "step", "type": "bf16", "batch": 256, "pool": 320,
         "heads_k": 8, "heads_v": 16, "dim_k": 128, "dim_v": 128, "idle": 13},
        # a short prompt that goes on from a kept state; q, k and v are slices of one projection
        {"name": "forward 100 from a state", "op": "forward", "type": "bf16", "lengths": "100", "packed": False,
         "fused": True, "state": True, "heads_k": 16, "heads_v": 32, "dim_k": 128, "dim_v": 128},
        # one long prompt: the chain over 128 chunks, with few heads beside it
        {"name": "forward 8192", "op": "forward", "type": "bf16", "lengths": "8192", "packed": False,
         "fused": False, "state": False, "heads_k": 16, "heads_v": 32, "dim_k": 128, "dim_v": 128},
        # prompts of a serving batch, packed: lengths from nothing to 1500
        {"name": "forward packed 16 prompts", "op": "forward", "type": "fp16",
         "lengths": "1500,1,64,700,0,63,65,333,128,1024,2,511,90,257,1200,31", "packed": True, "fused": False,
         "state": True, "heads_k": 8, "heads_v": 8, "dim_k": 64, "dim_v": 128},
        # the training shape of the CfC cell (256 rows of 64 steps, width 128) with its float32 values
        {"name": "backward 256 x 64 fp32", "op": "backward", "type": "fp32", "lengths": "64*256", "packed": False,
         "fused": False, "state": True, "heads_k": 1, "heads_v": 1, "dim_k": 128, "dim_v": 128},
        # a training step's micro-batch
        {"name": "backward 4 x 2048", "op": "backward", "type": "bf16", "lengths": "2048*4", "packed": False,
         "fused": False, "state": False, "heads_k": 8, "heads_v": 16, "dim_k": 128, "dim_v": 128},
        # documents packed for training, head widths that are no powers of two
        {"name": "backward packed 9 odd", "op": "backward", "type": "bf16",
         "lengths": "77,1000,1,640,333,64,0,129,812", "packed": True, "fused": True, "state": True, "heads_k": 3,
         "heads_v": 6, "dim_k": 96, "dim_v": 80},
        # the norm before a decode step's 8-bit products
        {"name": "norm e4m3 32 x 4096", "op": "norm_e4m3", "type": "bf16", "rows": 32, "width": 4096,
         "residual": "same", "group": 128},
        # the norm of a prompt or a training step, with the residual stream
        {"name": "norm 16384 x 4096", "op": "norm", "type": "bf16", "rows": 16384, "width": 4096,
         "residual": "same"},
        # its gradients, the residual stream's gradient added
        {"name": "norm backward 16384 x 4096", "op": "norm_backward", "type": "bf16", "rows": 16384,
         "width": 4096, "stream": True},
        # the norm of each head's output (rows of one head's width), odd row count
        {"name": "norm backward 99991 x 128", "op": "norm_backward", "type": "bf16", "rows": 99991,
         "width": 128, "stream": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "forward", "forward", "backward", "backward", "norm", "norm_e4m3", "norm_backward"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op.startswith("norm"):
        rows, width = _log_int(rng, 1, 16384), _log_int(rng, 1, 8192)
        if rng.random() < 0.5:
            width = -(-width // 8) * 8
        while rows * width > 1 << 26:
            rows //= 2
        case = {"op": op, "type": kind, "rows": rows, "width": width}
        if op == "norm_backward":
            case["stream"] = rng.random() < 0.5
        else:
            case["residual"] = rng.choice(["none", "same", "fp32"])
        if op == "norm_e4m3":
            case["group"] = rng.choice([0, 32, 64, 128])
        return case
    heads_k = rng.choice([1, 2, 3, 4, 8])
    case = {"op": op, "type": kind, "heads_k": heads_k, "heads_v": heads_k * rng.choice([1, 1, 2, 3]),
            "dim_k": rng.choice([16, 64, 96, 128, 128, rng.randint(1, 128)]),
            "dim_v": rng.choice([16, 64, 80, 128, 128, rng.randint(1, 256)])}
    if op == "step":
        batch = _log_int(rng, 1, 256)
        case.update(batch=batch, pool=batch + rng.randint(0, 64), idle=rng.randint(0, batch // 4))
        return case
    count = _log_int(rng, 1, 24)
    most = 4096 if op == "forward" else 2048
    if rng.random() < 0.5:
        length = _log_int(rng, 1, most)
        lengths = [length] * max(1, min(count, 60000 // (length * case["heads_v"])))
        case.update(lengths="%d*%d" % (length, len(lengths)), packed=False)
    else:
        lengths, room = [], 60000 // case["heads_v"]
        for _ in range(count):
            n = 0 if rng.random() < 0.1 else _log_int(rng, 1, min(most, 1500))
            n = min(n, room)
            room -= n
            lengths.append(n)
        lengths[0] = max(1, lengths[0])
        case.update(lengths=",".join(map(str, lengths)), packed=True)
    case.update(fused=rng.random() < 0.4, state=rng.random() < 0.5)
    return case


def _lengths(case):
    if "*" in case["lengths"]:
        n, count = case["lengths"].split("*")
        return [int(n)] * int(count)
    return [int(n) for n in case["lengths"].split(",")]


# ------------------------------------------------------------------- the inputs
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev, dtype=torch.float32)

    s = {"case": case}
    if case["op"].startswith("norm"):
        rows, width = case["rows"], case["width"]
        s["weight"] = (1 + 0.2 * normal(width)).to(dtype)
        if case["op"] == "norm_backward":
            h = 1.5 * normal(rows, width)
            s["h"] = h.to(dtype)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + EPS)
            s["grad_y"] = normal(rows, width).to(dtype)
            s["grad_h"] = normal(rows, width).to(dtype) if case["stream"] else None
        else:
            s["x"] = normal(rows, width).to(dtype)
            kind = case["residual"]
            s["residual"] = None if kind == "none" else normal(rows, width).to(dtype if kind == "same" else torch.float32)
        return s

    hk, hv, dk, dv = (case[n] for n in ("heads_k", "heads_v", "dim_k", "dim_v"))
    scale = dk ** -0.5

    def gates(*lead):
        # decays from a thousandth to about two a token, and gates all over (0, 1)
        rate = torch.exp(math.log(1e-3) + uniform(hv) * math.log(2e3))
        return -rate * (0.5 + uniform(*lead, hv)), torch.sigmoid(normal(*lead, hv))

    def unit(t):
        return t / t.norm(dim=-1, keepdim=True).clamp_min(1e-6)

    if case["op"] == "step":
        b, pool = case["batch"], case["pool"]
        s.update(q=unit(normal(b, hk, dk)).to(dtype), k=unit(normal(b, hk, dk)).to(dtype), v=normal(b, hv, dv).to(dtype))
        s["g"], s["beta"] = gates(b)
        s["pool"] = normal(pool, hv, dk, dv) * 0.3
        if pool == 1:
            s["slots"] = None
        else:
            slots = torch.randperm(pool, generator=gen, device=dev)[:b].to(torch.int32)
            if case["idle"]:
                slots[torch.randperm(b, generator=gen, device=dev)[:case["idle"]]] = -1
            s["slots"] = slots
        s["scale"] = scale
        return s

    lens = _lengths(case)
    lead = (sum(lens),) if case["packed"] else (len(lens), lens[0])
    if case["fused"]:
        # one projection's output, each part normalised where it lies
        row = torch.empty(*lead, 2 * hk * dk + hv * dv, device=dev, dtype=dtype)
        q = row[..., :hk * dk].unflatten(-1, (hk, dk))
        k = row[..., hk * dk:2 * hk * dk].unflatten(-1, (hk, dk))
        v = row[..., 2 * hk * dk:].unflatten(-1, (hv, dv))
    else:
        q, k = (torch.empty(*lead, hk, dk, device=dev, dtype=dtype) for _ in range(2))
        v = torch.empty(*lead, hv, dv, device=dev, dtype=dtype)
    q.copy_(unit(normal(*lead, hk, dk)))
    k.copy_(unit(normal(*lead, hk, dk)))
    v.copy_(normal(*lead, hv, dv))
    s.update(q=q, k=k, v=v, scale=scale, lens=lens)
    s["g"], s["beta"] = gates(*lead)
    s["offsets"] = None
    if case["packed"]:
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=dev)
    s["initial"] = normal(len(lens), hv, dk, dv) * 0.3 if case["state"] else None
    if case["op"] == "backward":
        s["grad_o"] = normal(*lead, hv, dv).to(dtype)
        s["grad_final"] = normal(len(lens), hv, dk, dv) * 0.1 if case["state"] else None
    return s


# -------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(op, s)
    if op == "step":
        return _plain_step(s)
    if op == "forward":
        return _plain_forward(s)
    if op == "backward":
        return _plain_backward(s)
    if op == "norm_backward":
        return _plain_norm_backward(s)
    return _plain_norm(s)


def _run_own(op, s):
    import cfc_recurrent_cell_amd as cfc
    if op == "step":
        o = cfc.delta_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], slots=s["slots"],
                                scale=s["scale"])
        return {"o": o, "pool": s["pool"]}
    if op == "forward":
        o, final = cfc.delta_rule_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], initial_state=s["initial"],
                                          scale=s["scale"], offsets=s["offsets"])
        return {"o": o, "final": final}
    if op == "backward":
        names = ("q", "k", "v", "g", "beta", "initial")
        grads = cfc.delta_rule_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["grad_o"],
                                        initial_state=s["initial"], grad_final_state=s["grad_final"],
                                        scale=s["scale"], offsets=s["offsets"])
        return dict(zip(names, grads))
    if op == "norm_backward":
        gx, gw = cfc.rms_norm_backward(s["grad_y"], s["h"], s["weight"], s["rstd"], grad_h=s["grad_h"])
        return {"x": gx, "weight": gw}
    if op == "norm_e4m3":
        y, scales, h = cfc.rms_norm_forward_e4m3(s["x"], s["weight"], EPS, residual=s["residual"],
                                                 group=s["case"]["group"])
        return {"y": y, "scales": scales, "h": h}
    y, h, rstd = cfc.rms_norm_forward(s["x"], s["weight"], EPS, residual=s["residual"])
    return {"y": y, "h": h, "rstd": rstd}


# ---------------------------------------------------- plain forms in 32 bits
def _plain_norm(s):
    case, x, w = s["case"], s["x"].float(), s["weight"].float()
    h = s["x"] if s["residual"] is None else (x + s["residual"].float()).to(s["residual"].dtype)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(-1) + EPS)
    y = hf * rstd[:, None] * w
    if case["op"] == "norm":
        return {"y": y.to(s["x"].dtype), "h": h, "rstd": rstd}
    rows, width = y.shape
    group = case["group"] or width
    groups = -(-width // group)
    padded = torch.zeros(rows, groups * group, device=y.device)
    padded[:, :width] = y
    padded = padded.view(rows, groups, group)
    amax = padded.abs().amax(-1)
    amax = torch.where(amax == 0, torch.ones_like(amax), amax)
    q = (padded * (448.0 / amax)[..., None]).reshape(rows, groups * group)[:, :width]
    return {"y": q.to(torch.float8_e4m3fn), "scales": amax / 448.0, "h": h}


def _plain_norm_backward(s):
    h, w, dy, rstd = s["h"].float(), s["weight"].float(), s["grad_y"].float(), s["rstd"][:, None]
    n = h * rstd
    dn = dy * w
    gx = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    if s["grad_h"] is not None:
        gx = gx + s["grad_h"].float()
    return {"x": gx.to(s["h"].dtype), "weight": (dy * n).sum(0, dtype=torch.float64).float()}


def _plain_step(s):
    case = s["case"]
    rep = case["heads_v"] // case["heads_k"]
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    o = torch.zeros_like(v)
    rows = torch.arange(case["batch"], device=v.device)
    at = rows if s["slots"] is None else s["slots"].long()
    rows = rows[at >= 0]
    at = at[at >= 0]
    q, k = q[rows].repeat_interleave(rep, 1), k[rows].repeat_interleave(rep, 1)
    S = s["pool"][at] * torch.exp(s["g"][rows])[..., None, None]
    u = s["beta"][rows][..., None] * (v[rows] - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    o[rows] = s["scale"] * (S * q[..., None]).sum(-2)
    s["pool"][at] = S
    return {"o": o.to(s["v"].dtype), "pool": s["pool"]}


def _places(s):
    """For each sequence and place in it, padded to whole chunks: the row of the packed tokens, and whether there is one."""
    lens = torch.tensor(s["lens"], device=s["q"].device)
    starts = lens.cumsum(0) - lens
    padded = max(1, -(-max(s["lens"]) // CHUNK)) * CHUNK
    place = torch.arange(padded, device=lens.device)
    there = place[None] < lens[:, None]
    return torch.where(there, starts[:, None] + place[None], torch.zeros_like(place)[None]), there


def _chunked(s, at, there, name, rep):
    """Input `name` in 32 bits as [sequence, value head, chunk, place, ...], zero where there is no token."""
    t = s[name]
    lead = 1 if s["offsets"] is not None else 2
    t = t.flatten(0, lead - 1).float()[at]
    t = torch.where(there.view(*there.shape, *([1] * (t.dim() - 2))), t, torch.zeros_like(t))
    t = t.repeat_interleave(rep, 2) if rep > 1 else t
    return t.transpose(1, 2).unflatten(2, (-1, CHUNK))


def _rows_of(s, t, at, there, like):
    """[sequence, head, chunk, place, ...] back to the token rows of `like`."""
    t = t.flatten(2, 3).transpose(1, 2)
    out = torch.zeros(int(sum(s["lens"])), *t.shape[2:], device=t.device)
    out[at[there]] = t[there]
    return out.view(*like.shape[:-1], *t.shape[3:]) if t.dim() == 4 else out.view(like.shape)


def _solved(s):
    """What the chunks of a sequence have before its states are known."""
    case = s["case"]
    rep = case["heads_v"] // case["heads_k"]
    at, there = _places(s)
    q, k = (_chunked(s, at, there, n, rep) for n in ("q", "k"))
    v, g, beta = (_chunked(s, at, there, n, 1) for n in ("v", "g", "beta"))
    G = g.double().cumsum(-1)  # sums of decays, of which only differences count
    one = torch.ones(CHUNK, CHUNK, device=q.device).tril()
    decay = torch.exp(torch.where(one > 0, G[..., :, None] - G[..., None, :], torch.zeros_like(one, dtype=torch.float64))).float() * one
    L = (beta[..., None] * decay * (k @ k.transpose(-1, -2))).tril(-1)
    inv = torch.eye(CHUNK, device=q.device).expand_as(L).clone()
    for i in range(1, CHUNK):
        inv[..., i, :i] = -(L[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    M = decay * (q @ k.transpose(-1, -2))
    begin = torch.exp(G).float()[..., None]
    end = torch.exp(G[..., -1:] - G).float()[..., None]
    first = s["initial"]
    if first is None:
        first = torch.zeros(q.shape[0], q.shape[1], case["dim_k"], case["dim_v"], device=q.device)
    return at, there, q, k, v, beta[..., None], decay, L, inv, M, begin, end, first


def _plain_forward(s):
    at, there, q, k, v, beta, decay, L, inv, M, begin, end, S = _solved(s)
    o = torch.empty_like(v)
    for c in range(q.shape[2]):
        u = inv[:, :, c] @ (beta[:, :, c] * (v[:, :, c] - begin[:, :, c] * (k[:, :, c] @ S)))
        o[:, :, c] = s["scale"] * (begin[:, :, c] * (q[:, :, c] @ S) + M[:, :, c] @ u)
        S = begin[:, :, c, -1:] * S + (end[:, :, c] * k[:, :, c]).transpose(-1, -2) @ u
    return {"o": _rows_of(s, o, at, there, s["v"]).to(s["v"].dtype), "final": S}


def _plain_backward(s):
    at, there, q, k, v, beta, decay, L, inv, M, begin, end, S = _solved(s)
    case, scale, chunks = s["case"], s["scale"], q.shape[2]
    do = _chunked(s, at, there, "grad_o", 1) * scale
    before, diffs, us = [], [], []
    for c in range(chunks):
        before.append(S)
        diffs.append(v[:, :, c] - begin[:, :, c] * (k[:, :, c] @ S))
        us.append(inv[:, :, c] @ (beta[:, :, c] * diffs[c]))
        S = begin[:, :, c, -1:] * S + (end[:, :, c] * k[:, :, c]).transpose(-1, -2) @ us[c]
    dS = torch.zeros_like(S) if s["grad_final"] is None else s["grad_final"]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dbeta, dG = torch.empty_like(beta), torch.empty_like(beta)
    for c in reversed(range(chunks)):
        qc, kc, b, S0, u, e = q[:, :, c], k[:, :, c], begin[:, :, c], before[c], us[c], end[:, :, c]
        du = M[:, :, c].transpose(-1, -2) @ do[:, :, c] + e * (kc @ dS)
        dr = inv[:, :, c].transpose(-1, -2) @ du
        dL = -(dr @ u.transpose(-1, -2)).tril(-1)
        dM = (do[:, :, c] @ u.transpose(-1, -2)).tril()
        db = beta[:, :, c] * dr
        E, F = dL * beta[:, :, c] * decay[:, :, c], dM * decay[:, :, c]
        from_S, at_S = b * (do[:, :, c] @ S0.transpose(-1, -2)), -b * (db @ S0.transpose(-1, -2))
        at_end = e * (u @ dS.transpose(-1, -2))
        dq[:, :, c] = from_S + F @ kc
        dk[:, :, c] = at_S + at_end + F.transpose(-1, -2) @ qc + (E + E.transpose(-1, -2)) @ kc
        dv[:, :, c] = db
        dbeta[:, :, c] = (dr * diffs[c]).sum(-1, keepdim=True) + (dL * decay[:, :, c] * (kc @ kc.transpose(-1, -2))).sum(-1, keepdim=True)
        D = dM * M[:, :, c] + dL * L[:, :, c]
        gone = (at_end * kc).sum(-1, keepdim=True)
        d = D.sum(-1, keepdim=True) - D.sum(-2)[..., None] + (from_S * qc + at_S * kc).sum(-1, keepdim=True) - gone
        d[..., -1:, :] += gone.sum(-2, keepdim=True) + b[..., -1:, :] * (dS * S0).sum((-1, -2))[..., None, None]
        dG[:, :, c] = d
        dS = b[..., -1:, :] * dS + (b * qc).transpose(-1, -2) @ do[:, :, c] - (b * kc).transpose(-1, -2) @ db
    dg = dG.double().flip(-2).cumsum(-2).flip(-2).float()  # a decay counts for all later places of its chunk
    rep = case["heads_v"] // case["heads_k"]
    dq, dk = (t.unflatten(1, (case["heads_k"], rep)).sum(2) for t in (dq, dk))
    out = {n: _rows_of(s, t, at, there, s[n]).to(s[n].dtype) for n, t in (("q", dq), ("k", dk), ("v", dv))}
    out["g"], out["beta"] = (_rows_of(s, t[..., 0], at, there, s["g"]) for t in (dg, dbeta))
    out["initial"] = dS if s["initial"] is not None else None
    return out


# ------------------------------------------- what the definition gives, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    if case["op"] == "step":
        return _exact_step(case, s)
    return _exact_sequence(case, s)


def _exact_norm(case, s):
    w = s["weight"].double()
    if case["op"] == "norm_backward":
        h, dy, rstd = s["h"].double(), s["grad_y"].double(), s["rstd"].double()[:, None]
        a = (dy * w * h).sum(-1, keepdim=True) / h.shape[-1]
        gx = dy * w * rstd - h * a * rstd ** 3
        if s["grad_h"] is not None:
            gx = gx + s["grad_h"].double()
        return {"x": gx, "weight": (dy * h * rstd).sum(0)}
    if s["residual"] is None:
        h = s["x"].double()
    else:  # the stream is kept in its own type, and the norm is that of what is kept
        h = (s["x"].double() + s["residual"].double()).to(s["residual"].dtype).double()
    rstd = 1 / torch.sqrt((h * h).sum(-1) / h.shape[-1] + EPS)
    y = h * w * rstd[:, None]
    if case["op"] == "norm":
        return {"y": y, "h": h, "rstd": rstd}
    group = case["group"] or case["width"]
    scales, parts = [], []
    for at in range(0, case["width"], group):
        part = y[:, at:at + group]
        top = part.abs().max(-1).values
        scale = torch.where(top > 0, top, torch.ones_like(top)) / 448
        scales.append(scale)
        parts.append(part / scale[:, None])
    return {"y": torch.cat(parts, 1), "scales": torch.stack(scales, 1), "h": h}


def _exact_step(case, s):
    rep = case["heads_v"] // case["heads_k"]
    pool = s["pool"].double()
    o = torch.zeros(case["batch"], case["heads_v"], case["dim_v"], dtype=torch.float64, device=pool.device)
    slots = list(range(case["batch"])) if s["slots"] is None else s["slots"].tolist()
    for b, at in enumerate(slots):
        if at < 0:
            continue
        k, q = (s[n][b].double().repeat_interleave(rep, 0) for n in ("k", "q"))
        S = pool[at] * s["g"][b].double().exp()[:, None, None]
        u = s["beta"][b].double()[:, None] * (s["v"][b].double() - torch.einsum("hkv,hk->hv", S, k))
        S = S + torch.einsum("hk,hv->hkv", k, u)
        pool[at] = S
        o[b] = s["scale"] * torch.einsum("hkv,hk->hv", S, q)
    return {"o": o, "pool": pool}


def _exact_sequence(case, s):
    lens, rep = s["lens"], case["heads_v"] // case["heads_k"]
    count, longest = len(lens), max(lens)
    dev = s["q"].device
    if count * longest * case["heads_v"] * case["dim_k"] * case["dim_v"] * 8 > 60e9 and case["op"] == "backward":
        return None

    def padded(t, heads):
        flat = t.double().reshape(-1, *t.shape[1 if case["packed"] else 2:])
        out = torch.zeros(longest, count, *flat.shape[1:], dtype=torch.float64, device=dev)
        start = 0
        for i, n in enumerate(lens):
            out[:n, i] = flat[start:start + n]
            start += n
        return out.repeat_interleave(heads, 2) if heads > 1 else out

    def packed(t, like):
        flat = torch.cat([t[:n, i] for i, n in enumerate(lens)])
        return flat.reshape(*like.shape[:1 if case["packed"] else 2], *flat.shape[1:])

    q, k = padded(s["q"], rep), padded(s["k"], rep)
    v, g, beta = padded(s["v"], 1), padded(s["g"], 1), padded(s["beta"], 1)
    S = torch.zeros(count, case["heads_v"], case["dim_k"], case["dim_v"], dtype=torch.float64, device=dev)
    if s["initial"] is not None:
        S = s["initial"].double()
    scale, decay = s["scale"], g.exp()
    back = case["op"] == "backward"
    states, errs, o = [], [], torch.zeros_like(v)
    for t in range(longest):
        S = S * decay[t][..., None, None]
        e = v[t] - (S * k[t][..., None]).sum(-2)
        if back:
            states.append(S)  # decayed, before the token's own correction
            errs.append(e)
        S = S + k[t][..., None] * (beta[t][..., None] * e)[..., None, :]
        if not back:
            o[t] = scale * (S * q[t][..., None]).sum(-2)
    if not back:
        return {"o": packed(o, s["v"]), "final": S}
    do = padded(s["grad_o"], 1)
    dS = torch.zeros_like(S) if s["grad_final"] is None else s["grad_final"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(g), torch.zeros_like(beta)
    for t in reversed(range(longest)):
        u = beta[t][..., None] * errs[t]
        after = states[t] + k[t][..., None] * u[..., None, :]
        dq[t] = scale * (after * do[t][..., None, :]).sum(-1)
        dS = dS + scale * q[t][..., None] * do[t][..., None, :]
        du = (dS * k[t][..., None]).sum(-2)
        de = beta[t][..., None] * du
        dbeta[t] = (du * errs[t]).sum(-1)
        dv[t] = de
        dk[t] = (dS * u[..., None, :]).sum(-1) - (states[t] * de[..., None, :]).sum(-1)
        dS = dS - k[t][..., None] * de[..., None, :]
        dg[t] = (dS * states[t]).sum((-1, -2))
        dS = dS * decay[t][..., None, None]
        states[t] = None
    dq, dk = (t.unflatten(2, (case["heads_k"], rep)).sum(3) for t in (dq, dk))
    out = {"q": packed(dq, s["q"]), "k": packed(dk, s["k"]), "v": packed(dv, s["v"]), "g": packed(dg, s["g"]),
           "beta": packed(dbeta, s["beta"])}
    out["initial"] = dS if s["initial"] is not None else None
    return out


# --------------------------------------------------------------------- the work
def work(case):
    size = BYTES[case["type"]]
    if case["op"].startswith("norm"):
        n, rows, width = case["rows"] * case["width"], case["rows"], case["width"]
        if case["op"] == "norm_backward":
            return {"bytes": n * size * (4 if case["stream"] else 3) + rows * 4 + width * (size + 4), "flops": 9 * n}
        h = {"none": 0, "same": 2 * size, "fp32": 8}[case["residual"]]
        if case["op"] == "norm":
            return {"bytes": n * (2 * size + h) + rows * 4 + width * size, "flops": 5 * n}
        groups = -(-width // (case["group"] or width))
        return {"bytes": n * (size + 1 + h) + rows * groups * 4 + width * size, "flops": 8 * n}
    hk, hv, dk, dv = (case[n] for n in ("heads_k", "heads_v", "dim_k", "dim_v"))
    state = hv * dk * dv
    token = 2 * hk * dk * size + hv * dv * size + 8 * hv
    if case["op"] == "step":
        b = case["batch"] - case["idle"]
        return {"bytes": b * (token + hv * dv * size + 8 * state), "flops": 7 * b * state}
    lens = _lengths(case)
    tokens, kept = sum(lens), len(lens) * state * 4
    if case["op"] == "forward":
        return {"bytes": tokens * (token + hv * dv * size) + kept * (2 if case["state"] else 1),
                "flops": 7 * tokens * state}
    # the states again, then the same products for their gradients
    return {"bytes": tokens * (2 * token + hv * dv * size) + (3 * kept if case["state"] else 0),
            "flops": 22 * tokens * state}
