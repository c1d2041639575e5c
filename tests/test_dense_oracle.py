"""The dense block's fp64 oracle: closed forms, gradients against differences (CPU)."""

import math

import numpy as np
import pytest

from oracle import dense_oracle as O

ACTS = ["none", "relu", "gelu_tanh", "silu"]


def _diff(f, x, dy, step=1e-6):
    """Central differences of sum(f(x) * dy) with respect to every element of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + step
        hi = (f(x) * dy).sum()
        x[i] = old - step
        lo = (f(x) * dy).sum()
        x[i] = old
        g[i] = (hi - lo) / (2 * step)
    return g


@pytest.mark.parametrize("kind", ACTS)
def test_derivative_against_differences(kind):
    z = np.concatenate([np.linspace(-6, 6, 41) + 0.013, [-50.0, 50.0, -200.0, 200.0]])
    d = (O.act(z + 1e-5, kind) - O.act(z - 1e-5, kind)) / 2e-5
    # the differences' own error: 1e-10 of curvature and 2^-53 |z| / 1e-5 of rounding
    assert (np.abs(d - O.dact(z, kind)) < 1e-8 + np.abs(z) * 1e-10).all()


def test_activations_by_hand():
    z = np.array([0.0, 1.0, -1.0, 3.0])
    t = np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    assert np.allclose(O.act(z, "gelu_tanh"), 0.5 * z * (1 + t), rtol=0, atol=1e-15)
    assert np.allclose(O.act(z, "silu"), z / (1 + np.exp(-z)), rtol=0, atol=1e-15)
    assert np.isnan(O.act(np.array([np.nan]), "silu")).all() and O.act(np.array([np.nan]), "relu")[0] == 0


@pytest.mark.parametrize("T,D", [(1, 1), (3, 5), (2, 8)])
def test_norm_gradients_against_differences(T, D):
    rng = np.random.default_rng(T + D)
    x, r, w, dy = rng.normal(size=(T, D)), rng.normal(size=(T, D)), rng.normal(size=D), rng.normal(size=(T, D))
    y, h, rstd = O.rms_norm(x, w, 1e-3, r)
    dx, dw = O.rms_norm_bwd(dy, h, w, rstd)
    assert np.allclose(dx, _diff(lambda v: O.rms_norm(v, w, 1e-3, r)[0], x, dy), atol=1e-7)
    assert np.allclose(dw, _diff(lambda v: O.rms_norm(x, v, 1e-3, r)[0], w, dy), atol=1e-7)
    dh = rng.normal(size=(T, D))
    assert np.allclose(O.rms_norm_bwd(dy, h, w, rstd, dh)[0], dx + dh)


def test_linear_gradients_against_differences():
    rng = np.random.default_rng(5)
    x, w, b, dy = rng.normal(size=(3, 4)), rng.normal(size=(5, 4)), rng.normal(size=5), rng.normal(size=(3, 5))
    for kind in ("gelu_tanh", "silu"):
        f = lambda v, m, c: O.linear(v, m, c, kind)[0]
        z = O.linear(x, w, b, kind)[1]
        dz = dy * O.dact(z, kind)
        assert np.allclose(dz @ w, _diff(lambda v: f(v, w, b), x, dy), atol=1e-7)
        assert np.allclose(dz.T @ x, _diff(lambda v: f(x, v, b), w, dy), atol=1e-7)
        assert np.allclose(dz.sum(0), _diff(lambda v: f(x, w, v), b, dy), atol=1e-7)


def test_scales_by_hand():
    y = np.zeros((1, 300))
    y[0, 3], y[0, 130], y[0, 299] = 448.0, 449.0, 1.75 * 2.0 ** -140
    s, near = O.scales(y, "e4m3")
    assert s[:, 0].tolist() == [1.0, 2.0, 2.0 ** -126] and near[:2, 0].tolist() == [True, False]
    assert O.scales(np.zeros((2, 5)), "e5m2")[0].tolist() == [[1.0, 1.0]]


def test_norm_of_gradients_by_hand():
    assert O.grad_norm([np.array([3.0]), np.array([[4.0], [12.0]])]) == 13.0
    assert O.grad_factor(13.0, 26.0) == 1.0 and O.grad_factor(13.0, 6.5) == 0.5
    assert O.grad_factor(math.inf, 1.0) == 1.0 and O.grad_factor(math.nan, 1.0) == 1.0
