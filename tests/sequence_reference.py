"""The selective scan, the short causal convolution and the layer norm in float64 on the
CPU, token by token, and their adjoints: the definitions that the library's kernels are held
to.  Written from the formulas alone; tests/test_sequence_reference.py holds the adjoints to
central differences.

With ``size=True`` the same sums are taken of magnitudes: what roundings are relative to."""
import numpy as np

from delta_rule_reference import spans  # noqa: F401


def sigmoid(x):
    return np.exp(-np.logaddexp(0.0, -x))


def silu_slope(x, size=False):
    s = sigmoid(x)
    return s * (1 + (np.abs(x) if size else x) * (1 - s))


# ------------------------------------------------------------------ the scan
NAMES = ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "initial")


def scan(p, rows, softplus=True, gy=None, gfinal=None, size=False):
    """(y, final, None), or with gy (y, final, gradients): p has x, dt [tokens, channels],
    a [channels, state], b, c [tokens, groups, state], initial [sequences, channels, state] and,
    or None, d, dt_bias [channels] and z [tokens, channels]."""
    mag = np.abs if size else np.asarray
    x, a, initial = mag(p["x"]), p["a"], mag(p["initial"])
    share = x.shape[1] // p["b"].shape[1]
    b, c = (np.repeat(mag(p[n]), share, 1) for n in ("b", "c"))
    d = np.zeros(x.shape[1]) if p["d"] is None else mag(p["d"])
    pre = p["dt"] + (0 if p["dt_bias"] is None else p["dt_bias"])
    step = np.logaddexp(0.0, pre) if softplus else pre
    slope = sigmoid(pre) if softplus else np.ones_like(pre)
    gate = np.ones_like(x) if p["z"] is None else mag(p["z"] * sigmoid(p["z"]))
    decay = np.exp(step[..., None] * a)
    step = mag(step)
    add = (step * x)[..., None] * b
    ypre, final, before = np.zeros_like(x), initial.copy(), np.zeros_like(decay)
    for i, (start, n) in enumerate(rows):
        h = initial[i].copy()
        for t in range(start, start + n):
            before[t] = h
            h = decay[t] * h + add[t]
            ypre[t] = (c[t] * h).sum(-1) + d * x[t]
        final[i] = h
    y = ypre * gate
    if gy is None:
        return y, final, None
    gy = mag(gy)
    g = {n: np.zeros_like(x) for n in ("x", "dt", "z")}
    g.update(a=np.zeros_like(a), b=np.zeros_like(b), c=np.zeros_like(b), initial=np.zeros_like(initial))
    if p["z"] is not None:
        g["z"] = gy * ypre * silu_slope(p["z"], size)
    gp = gy * gate
    for i, (start, n) in enumerate(rows):
        e = mag(gfinal[i]).copy()
        for t in reversed(range(start, start + n)):
            h = decay[t] * before[t] + add[t]
            e = e + gp[t][:, None] * c[t]
            g["c"][t] = gp[t][:, None] * h
            g["b"][t] = e * (step[t] * x[t])[:, None]
            into = e * decay[t] * before[t]
            gu = (e * b[t]).sum(-1)
            g["x"][t] = gu * step[t] + d * gp[t]
            g["dt"][t] = (gu * x[t] + (into * mag(a)).sum(-1)) * slope[t]
            g["a"] += into * step[t][:, None]
            e = decay[t] * e
        g["initial"][i] = e
    for n in ("b", "c"):
        g[n] = g[n].reshape(*p["b"].shape[:2], share, -1).sum(2)
    g["d"] = (gp * x).sum(0)
    g["dt_bias"] = g["dt"].sum(0)
    return y, final, g


def scan_inputs(gen, tokens, sequences, channels, groups, state, gated=True):
    """Steps from a thousandth to a few, decays from none to nearly all."""
    n = gen.standard_normal
    return {"x": n((tokens, channels)), "dt": 1.5 * n((tokens, channels)), "a": -np.exp(n((channels, state))),
            "b": n((tokens, groups, state)), "c": n((tokens, groups, state)), "d": 1 + 0.3 * n(channels),
            "z": n((tokens, channels)) if gated else None, "dt_bias": -2 + n(channels),
            "initial": 0.5 * n((sequences, channels, state))}


# ----------------------------------------------------------- the convolution
def conv(x, w, bias, initial, rows, silu=True, gy=None, gfinal=None, size=False):
    """(y, final, None), or with gy (y, final, gradients): x [tokens, channels], w
    [channels, width], initial [sequences, width - 1, channels], bias [channels] or None."""
    mag = np.abs if size else np.asarray
    width = w.shape[1]
    xs, ws, bs = mag(x), mag(w), mag(np.zeros(x.shape[1]) if bias is None else bias)
    y, final = np.zeros_like(x), np.zeros_like(initial)
    g = {"x": np.zeros_like(x), "weight": np.zeros_like(w), "bias": np.zeros(x.shape[1]), "initial": np.zeros_like(initial)}
    for i, (start, n) in enumerate(rows):
        seen, raw = (np.concatenate([k, m[start:start + n]]) for k, m in ((mag(initial[i]), xs), (initial[i], x)))
        p, true = (np.zeros((n, x.shape[1])) + k for k in (bs, 0 if bias is None else bias))
        for j in range(width):
            p = p + seen[j:j + n] * ws[:, j]
            true = true + raw[j:j + n] * w[:, j]
        # p's own error, relative to its terms' magnitudes, goes on with y'(p), or y''(p) in a gradient
        slope, curve = silu_slope(true, size), 0.0
        if size and silu:
            s = sigmoid(true)
            curve = s * (1 - s) * (2 + np.abs(true * (1 - 2 * s))) * p
        y[start:start + n] = (p * slope if size else p * sigmoid(true)) if silu else p
        final[i] = seen[n:]
        if gy is None:
            continue
        gp = mag(gy[start:start + n]) * (slope + curve if silu else 1)
        gs = np.zeros_like(seen)
        for j in range(width):
            gs[j:j + n] += gp * ws[:, j]
            g["weight"][:, j] += (gp * seen[j:j + n]).sum(0)
        gs[n:] += mag(gfinal[i])
        g["bias"] += gp.sum(0)
        g["initial"][i] = gs[:width - 1]
        g["x"][start:start + n] = gs[width - 1:]
    return y, final, None if gy is None else g


# ------------------------------------------------------------- the layer norm
def layer_norm(h, w, bias, eps):
    mean = h.mean(-1)
    rstd = 1 / np.sqrt(((h - mean[:, None]) ** 2).mean(-1) + eps)
    return (h - mean[:, None]) * rstd[:, None] * w + bias, mean, rstd


def layer_norm_backward(gy, h, w, mean, rstd):
    n = (h - mean[:, None]) * rstd[:, None]
    d = gy * w
    gx = rstd[:, None] * (d - d.mean(-1, keepdims=True) - n * (d * n).mean(-1, keepdims=True))
    return gx, (gy * n).sum(0), gy.sum(0)
