"""The float64 references of the scan, the convolution and the layer norm: their adjoints
against central differences, and identities."""
import numpy as np
import pytest

import sequence_reference as R

STEP = 1e-5  # error of the difference about STEP^2 + 2^-53 / STEP, 1e-10 and 1e-11 of the value's terms


def differences(value, args, grads, size=1.0):
    """``size``: the magnitudes of the value's terms, summed."""
    for name, got in grads.items():
        want = np.zeros_like(got)
        for at in np.ndindex(*got.shape):
            side = []
            for sign in (1, -1):
                y = {n: None if v is None else v.copy() for n, v in args.items()}
                y[name][at] += sign * STEP
                side.append(value(y))
            want[at] = (side[0] - side[1]) / (2 * STEP)
        np.testing.assert_allclose(got, want, rtol=1e-7, atol=2e-8 * max(1.0, size), err_msg=name)


@pytest.mark.parametrize("groups,state,lens,softplus,gated", [(1, 3, [5], True, True), (2, 2, [3, 0, 1, 4], True, False),
                                                              (1, 1, [2, 2], False, True)])
def test_scan_adjoint_matches_central_differences(groups, state, lens, softplus, gated):
    gen = np.random.default_rng(3)
    rows, tokens = R.spans(lens), sum(lens)
    p = R.scan_inputs(gen, tokens, len(lens), 2 * groups, groups, state, gated)
    gy, gf = gen.standard_normal((tokens, 2 * groups)), gen.standard_normal((len(lens), 2 * groups, state))

    def value(q):
        y, final, _ = R.scan(q, rows, softplus)
        return (y * gy).sum() + (final * gf).sum()

    y, final, g = R.scan(p, rows, softplus, gy, gf)
    differences(value, p, {n: g[n] for n in R.NAMES if p[n] is not None}, np.abs(y * gy).sum() + np.abs(final * gf).sum())


@pytest.mark.parametrize("width,lens,silu,bias", [(4, [6], True, True), (3, [3, 0, 1, 4], True, False), (2, [2, 1], False, True)])
def test_conv_adjoint_matches_central_differences(width, lens, silu, bias):
    gen = np.random.default_rng(4)
    rows, tokens, n = R.spans(lens), sum(lens), gen.standard_normal
    p = {"x": n((tokens, 2)), "weight": n((2, width)), "bias": n(2) if bias else None, "initial": n((len(lens), width - 1, 2))}
    gy, gf = n((tokens, 2)), n((len(lens), width - 1, 2))

    def value(q):
        y, final, _ = R.conv(q["x"], q["weight"], q["bias"], q["initial"], rows, silu)
        return (y * gy).sum() + (final * gf).sum()

    _, _, g = R.conv(p["x"], p["weight"], p["bias"], p["initial"], rows, silu, gy, gf)
    differences(value, p, {k: g[k] for k in p if p[k] is not None})


def test_layer_norm_adjoint_matches_central_differences():
    gen = np.random.default_rng(5)
    p = {"h": gen.standard_normal((3, 5)) + 2, "w": gen.standard_normal(5), "b": gen.standard_normal(5)}
    gy = gen.standard_normal((3, 5))
    _, mean, rstd = R.layer_norm(p["h"], p["w"], p["b"], 1e-2)
    gx, gw, gb = R.layer_norm_backward(gy, p["h"], p["w"], mean, rstd)
    differences(lambda q: (R.layer_norm(q["h"], q["w"], q["b"], 1e-2)[0] * gy).sum(), p, {"h": gx, "w": gw, "b": gb})


def test_a_step_of_nothing_leaves_the_state():
    gen = np.random.default_rng(6)
    p = R.scan_inputs(gen, 3, 1, 4, 1, 5)
    p["dt"][:] = 0
    p["dt_bias"][:] = 0
    _, final, _ = R.scan(p, R.spans([3]), softplus=False)
    np.testing.assert_array_equal(final, p["initial"])


def test_a_sequence_in_two_halves_is_the_whole():
    gen = np.random.default_rng(7)
    p = R.scan_inputs(gen, 7, 1, 4, 2, 3)
    y, final, _ = R.scan(p, R.spans([7]))
    parts, state = [], p["initial"]
    for lo, hi in ((0, 3), (3, 7)):
        q = {n: v[lo:hi] if n in ("x", "dt", "b", "c", "z") else v for n, v in p.items()}
        out, state, _ = R.scan({**q, "initial": state}, R.spans([hi - lo]))
        parts.append(out)
    np.testing.assert_array_equal(np.concatenate(parts), y)
    np.testing.assert_array_equal(state, final)
    w, b, k = gen.standard_normal((4, 3)), gen.standard_normal(4), gen.standard_normal((1, 2, 4))
    y, final, _ = R.conv(p["x"], w, b, k, R.spans([7]))
    first, state, _ = R.conv(p["x"][:1], w, b, k, R.spans([1]))
    rest, state, _ = R.conv(p["x"][1:], w, b, state, R.spans([6]))
    np.testing.assert_array_equal(np.concatenate([first, rest]), y)
    np.testing.assert_array_equal(state, final)
