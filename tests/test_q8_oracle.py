"""The oracle of rows in 8 bits against brute force, closed forms and differences."""
import math

import numpy as np
import pytest

from oracle import q8_oracle as qo


@pytest.mark.parametrize("pow2", [True, False])
def test_codes_are_the_nearest_whole_numbers(pow2):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 33)) * np.exp(4 * rng.standard_normal((40, 1)))).astype(np.float32).astype(np.float64)
    q, s = qo.quantize_rows(x, pow2=pow2)
    grid = np.arange(-127, 128)
    for t in range(40):
        off = np.abs(x[t][:, None] - grid * s[t])
        assert (np.abs(x[t] - q[t] * s[t]) <= off.min(1) * (1 + 1e-12)).all()
        if pow2:
            assert math.frexp(s[t])[0] == 0.5 and 127 * s[t] >= np.abs(x[t]).max() > 127 * s[t] / 2
        else:
            assert s[t] == np.float32(np.abs(x[t]).max().astype(np.float32) / np.float32(127))


def test_ties_limits_and_special_rows():
    s = 2.0 ** -3
    x = np.array([[127 * s, 0.5 * s, 1.5 * s, 2.5 * s, -0.5 * s, -2.5 * s, -3.5 * s]])
    q, scale = qo.quantize_rows(x)
    assert scale[0] == s and q[0].tolist() == [127, 0, 2, 2, 0, -2, -4]
    q, scale = qo.quantize_rows(np.array([[127 * s * (1 + 2.0 ** -23), 0.0]]))
    assert scale[0] == 2 * s and q[0, 0] == 64
    special = np.array([[np.inf, 1], [np.nan, 1], [0, 0], [1, 2], [2.0 ** -140, 0], [3.4e38, 0]])
    q, scale = qo.quantize_rows(special, mask=[1, 1, 1, 0, 1, 1])
    assert np.isnan(scale[:2]).all() and scale[2] == 1 and scale[3] == 0 and scale[4] == 2.0 ** -126
    assert scale[5] == 2.0 ** 122 and q[5, 0] == 63
    assert not q[:5].any()


def test_products_by_elements():
    rng = np.random.default_rng(2)
    q, s = rng.integers(-127, 128, (7, 5)), np.array([1, 2, 0, 0.5, 4, 0, 1.0])
    g, w, v = rng.standard_normal((7, 3)), rng.integers(-127, 128, (3, 5)), rng.random(3)
    dw, db, size, _ = qo.weight_grad(g, q, s)
    y, _ = qo.linear(q, s, w, v, np.arange(3))
    for o in range(3):
        assert abs(db[o] - sum(g[t, o] for t in (0, 1, 3, 4, 6))) < 1e-12
        for k in range(5):
            assert abs(dw[o, k] - sum(g[t, o] * s[t] * q[t, k] for t in range(7))) < 1e-9
        for t in range(7):
            assert abs(y[t, o] - (sum(int(q[t, k]) * int(w[o, k]) for k in range(5)) * s[t] * v[o] + o)) < 1e-9
    packed, _ = qo.factor_packed(q, s, True)
    a = np.concatenate([q * s[:, None], np.ones((7, 1))], 1)
    want = [sum(a[t, i] * a[t, j] for t in (0, 1, 3, 4, 6)) / 5 for i in range(6) for j in range(i, 6)]
    assert np.allclose(packed, want, rtol=1e-12)
    assert packed[-1] == 1.0
    assert (qo.factor_packed(q, 0 * s, True)[0] == 0).all()
    assert (qo.factor_packed(q, 0 * s, True, old=packed, decay=0.9)[0] == packed).all()


def test_weight_gradient_against_differences():
    """d/dW of sum(c * y) with y the values times W^T plus b, by central differences: both are linear in W."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((9, 4))
    q, s = qo.quantize_rows(x, mask=[1] * 8 + [0])
    c, W, b = rng.standard_normal((9, 3)), rng.standard_normal((3, 4)), rng.standard_normal(3)

    def f(W, b):
        return float((c * (qo.row_values(q, s) @ W.T + b))[s != 0].sum())

    dw, db, _, _ = qo.weight_grad(c, q, s)
    h = 0.5
    for o in range(3):
        e = np.eye(3)[o] * h
        assert abs((f(W, b + e) - f(W, b - e)) / (2 * h) - db[o]) < 1e-11
        for k in range(4):
            E = np.zeros_like(W)
            E[o, k] = h
            assert abs((f(W + E, b) - f(W - E, b)) / (2 * h) - dw[o, k]) < 1e-11
