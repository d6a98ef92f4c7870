"""The float64 reference of the gated delta rule: its adjoint against central
differences, and identities of the recurrence."""
import numpy as np
import pytest

import delta_rule_reference as R


@pytest.mark.parametrize("hk,hv,lens", [(1, 1, [5]), (2, 4, [3, 0, 1, 4])])
def test_adjoint_matches_central_differences(hk, hv, lens):
    rows = R.spans(lens)
    x = R.inputs(3, rows, sum(lens), hk, hv, 3, 2)
    scale = 0.7

    def value(y):
        o, final, _ = R.forward(y["q"], y["k"], y["v"], y["g"], y["beta"], y["s0"], scale, rows)
        return (o * x["go"]).sum() + (final * x["gfinal"]).sum()

    grads, _ = R.backward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], scale, rows, x["go"], x["gfinal"])
    step = 1e-5  # error of the difference about step^2 + 2^-53 / step, 1e-10 and 1e-11 of the value
    for name, key in (("q", "q"), ("k", "k"), ("v", "v"), ("g", "g"), ("beta", "beta"), ("s0", "initial")):
        got = grads[key]
        want = np.zeros_like(got)
        for at in np.ndindex(*got.shape):
            side = []
            for sign in (1, -1):
                y = {n: a.copy() for n, a in x.items()}
                y[name][at] += sign * step
                side.append(value(y))
            want[at] = (side[0] - side[1]) / (2 * step)
        np.testing.assert_allclose(got, want, rtol=1e-7, atol=1e-8, err_msg=name)


def test_a_gate_of_one_stores_the_value_for_a_unit_key():
    rows = R.spans([1])
    x = R.inputs(5, rows, 1, 1, 1, 8, 4)
    k = x["k"] / np.linalg.norm(x["k"])
    _, final, _ = R.forward(x["q"], k, x["v"], x["g"], np.ones((1, 1)), x["s0"], 1.0, rows)
    np.testing.assert_allclose(final[0, 0].T @ k[0, 0], x["v"][0, 0], rtol=1e-12)


def test_total_decay_forgets():
    rows = R.spans([2])
    x = R.inputs(6, rows, 2, 1, 2, 4, 3)
    x["g"][1] = -np.inf
    o, final, _ = R.forward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], 1.0, rows)
    o1, final1, _ = R.forward(x["q"][1:], x["k"][1:], x["v"][1:], np.zeros_like(x["g"][1:]), x["beta"][1:], 0 * x["s0"], 1.0,
                              R.spans([1]))
    np.testing.assert_array_equal(final, final1)
    np.testing.assert_array_equal(o[1], o1[0])
