"""The gated delta rule token by token in float64 on the CPU, and its adjoint:
the definition that the library's chunked kernels are held to.  Written from
the recurrence alone; tests/test_delta_rule_reference.py holds the adjoint to
central differences."""
import numpy as np


def spans(lens=None, batch=None, length=None):
    """(first row, rows) of each sequence, packed or all of one length."""
    if lens is None:
        return [(b * length, length) for b in range(batch)]
    out, at = [], 0
    for n in lens:
        out.append((at, n))
        at += n
    return out


def forward(q, k, v, g, beta, s0, scale, rows):
    """o [tokens, heads_v, dim_v], S [sequences, heads_v, dim_k, dim_v] and what the
    adjoint reads.  q, k [tokens, heads_k, dim_k]; all float64."""
    rep = v.shape[1] // q.shape[1]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    o, final, kept = np.zeros_like(v), np.array(s0), {}
    with np.errstate(invalid="ignore"):
        decay = np.exp(g)
    for i, (start, n) in enumerate(rows):
        s = np.array(s0[i])
        for t in range(start, start + n):
            s = s * decay[t][:, None, None]
            err = v[t] - np.einsum("hkv,hk->hv", s, k[t])
            kept[t] = (s, err)
            s = s + k[t][:, :, None] * (beta[t][:, None] * err)[:, None, :]
            o[t] = scale * np.einsum("hkv,hk->hv", s, q[t])
        final[i] = s
    return o, final, kept


def backward(q, k, v, g, beta, s0, scale, rows, go, gfinal):
    """Gradients of sum(o go) + sum(final gfinal), and for each token and head the
    sum of the magnitudes that grad_g is the signed sum of."""
    rep = v.shape[1] // q.shape[1]
    _, _, kept = forward(q, k, v, g, beta, s0, scale, rows)
    hk = q.shape[1]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    gq, gk, gv, gg, gb = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(g), np.zeros_like(beta)
    mag = np.zeros_like(g)
    gs0 = np.array(gfinal)
    for i, (start, n) in enumerate(rows):
        ds = np.array(gfinal[i])
        for t in reversed(range(start, start + n)):
            s, err = kept[t]
            u = beta[t][:, None] * err
            after = s + k[t][:, :, None] * u[:, None, :]
            gq[t] = scale * np.einsum("hkv,hv->hk", after, go[t])
            ds = ds + scale * q[t][:, :, None] * go[t][:, None, :]
            du = np.einsum("hkv,hk->hv", ds, k[t])
            derr = beta[t][:, None] * du
            gb[t] = (du * err).sum(-1)
            gv[t] = derr
            gk[t] = np.einsum("hkv,hv->hk", ds, u) - np.einsum("hkv,hv->hk", s, derr)
            ds = ds - k[t][:, :, None] * derr[:, None, :]
            gg[t] = (ds * s).sum((-1, -2))
            mag[t] = np.abs(ds * s).sum((-1, -2)) + np.abs(gq[t] * q[t]).sum(-1) + np.abs(gk[t] * k[t]).sum(-1)
            ds = ds * np.exp(g[t])[:, None, None]
        gs0[i] = ds
    gq, gk = (x.reshape(x.shape[0], hk, rep, -1).sum(2) for x in (gq, gk))
    return {"q": gq, "k": gk, "v": gv, "g": gg, "beta": gb, "initial": gs0}, mag


def inputs(seed, rows, tokens, hk, hv, dk, dv, state=True, rate=1.0, beta_top=1.0, k_norm=True):
    """Float64 inputs whose values are also float32 values."""
    r = np.random.default_rng(seed)
    x = {"q": r.standard_normal((tokens, hk, dk)), "k": r.standard_normal((tokens, hk, dk)),
         "v": r.standard_normal((tokens, hv, dv)), "go": r.standard_normal((tokens, hv, dv)),
         "g": -rate * r.random((tokens, hv)) * np.exp(r.uniform(-3, 1, hv)), "beta": beta_top * r.random((tokens, hv)),
         "s0": 0.3 * r.standard_normal((len(rows), hv, dk, dv)), "gfinal": 0.3 * r.standard_normal((len(rows), hv, dk, dv))}
    if not state:
        x["s0"][:] = 0
        x["gfinal"][:] = 0
    if k_norm:
        x["k"] /= np.linalg.norm(x["k"], axis=-1, keepdims=True)
        x["q"] /= np.linalg.norm(x["q"], axis=-1, keepdims=True)
    return {n: a.astype(np.float32).astype(np.float64) for n, a in x.items()}
