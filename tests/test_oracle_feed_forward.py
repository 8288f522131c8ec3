"""Pins of the feed-forward oracle: closed forms, limits, and every gradient
against central differences of the value it belongs to."""

import numpy as np
import pytest

from oracle import feed_forward as ff

ACTS = ["none", "relu", "silu", "gelu"]


def test_norm_closed_forms():
    w = np.array([1.0, -2.0, 0.5, 3.0])
    y, r = ff.rms_norm([[3.0, 3.0, 3.0, 3.0], [0.0, -8.0, 0.0, 0.0], [0.0, 0.0, 0.0, 0.0]], w, 0.0 + 1e-30)
    assert np.allclose(r[:2], [1 / 3.0, 1 / 4.0], rtol=1e-14)      # rms of a constant row; of one nonzero in four
    assert np.allclose(y[0], w, rtol=1e-14) and np.allclose(y[1], [0, 4.0, 0, 0], rtol=1e-14)
    assert np.all(y[2] == 0) and np.isclose(r[2], 1e15)
    # eps adds to the mean square: 4 + 5 = 9
    assert np.isclose(ff.rms_norm([[2.0, 2.0]], [1.0, 1.0], 5.0)[1][0], 1 / 3.0, rtol=1e-15)


def test_activation_limits_and_forms():
    z = np.linspace(-6, 6, 241)
    for act in ACTS:
        v, _ = ff.activation(z, act)
        assert ff.activation(0.0, act)[0] == 0.0
        if act != "none":
            assert abs(ff.activation(30.0, act)[0] - 30.0) < 1e-11 and abs(ff.activation(-40.0, act)[0]) < 1e-14
    assert np.allclose(ff.activation(z, "silu")[0], 0.5 * z * (1 + np.tanh(z / 2)), atol=1e-14)
    u = ff.C * (z + ff.A * z ** 3)
    assert np.allclose(ff.activation(z, "gelu")[0], z / (1 + np.exp(-2 * u)), atol=1e-13)
    assert ff.activation(1.0, "gelu")[0] == pytest.approx(0.8411919906, abs=1e-9)


@pytest.mark.parametrize("act", ACTS)
def test_activation_slopes_against_differences(act):
    z = np.concatenate([np.linspace(-8, 8, 161) + 0.013, [-30.0, 30.0]])
    e = 1e-5
    num = (ff.activation(z + e, act)[0] - ff.activation(z - e, act)[0]) / (2 * e)
    assert np.allclose(ff.activation(z, act)[1], num, atol=1e-9)


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(3)
    h, w, dy = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7))
    dh, dw = ff.rms_norm_grad(dy, h, w, 0.1)
    e = 1e-6
    for i in range(3):
        for j in range(7):
            d = np.zeros_like(h)
            d[i, j] = e
            num = np.sum(dy * (ff.rms_norm(h + d, w, 0.1)[0] - ff.rms_norm(h - d, w, 0.1)[0])) / (2 * e)
            assert dh[i, j] == pytest.approx(num, abs=1e-8)
    for j in range(7):
        d = np.zeros(7)
        d[j] = e
        num = np.sum(dy * (ff.rms_norm(h, w + d, 0.1)[0] - ff.rms_norm(h, w - d, 0.1)[0])) / (2 * e)
        assert dw[j] == pytest.approx(num, abs=1e-8)


@pytest.mark.parametrize("act", ACTS)
def test_gated_gradient_against_differences(act):
    rng = np.random.default_rng(5)
    g, u, dh = rng.normal(size=50) * 2 + 0.01, rng.normal(size=50), rng.normal(size=50)
    dg, du = ff.gated_grad(dh, g, u, act)
    e = 1e-6
    assert np.allclose(dg, dh * (ff.gated(g + e, u, act) - ff.gated(g - e, u, act)) / (2 * e), atol=1e-8)
    assert np.allclose(du, dh * (ff.gated(g, u + e, act) - ff.gated(g, u - e, act)) / (2 * e), atol=1e-8)
