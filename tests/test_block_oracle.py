"""Pins of the float64 oracle of the operators around the projections: its
gradients against central differences, closed forms and invariants (CPU)."""

import math

import numpy as np
import pytest

from oracle import block_oracle as bo

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
H = 1e-6  # central differences: error H^2 f''' / 6 + 2^-53 |f| / H, about 1e-9


def difference(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        x[i] += H
        up = f()
        x[i] -= 2 * H
        g[i] = (up - f()) / (2 * H)
        x[i] += H
    return g


@pytest.mark.parametrize("name", ACTS)
def test_linear_gradients_are_differences(name):
    rng = np.random.default_rng(1)
    x, W = rng.standard_normal((3, 4)), rng.standard_normal((5, 4))
    bias, res = rng.standard_normal(5), rng.standard_normal((3, 5))
    dy = rng.standard_normal((3, 5))
    loss = lambda: float((dy * bo.linear(x, W, bias, res, name)[0]).sum())  # noqa: E731
    _, z = bo.linear(x, W, bias, res, name)
    assert np.abs(z).min() > 10 * H  # no step across relu's corner
    dx, dbias, _ = bo.linear_backward(dy, z, W, name)
    for got, arr in ((dx, x), (dbias, bias), (dy, res)):
        assert np.abs(got - difference(loss, arr)).max() < 1e-7


def test_activation_values():
    z = np.array([-1.0, 0.0, 2.0])
    assert np.allclose(bo.act(z, "relu"), [0, 0, 2])
    assert np.allclose(bo.act(z, "silu"), [-1 / (1 + math.e), 0, 2 / (1 + math.exp(-2))])
    # Phi(2) = 0.977249868051821 (standard normal table)
    assert abs(bo.act(z, "gelu")[2] - 2 * 0.977249868051821) < 1e-14
    assert abs(bo.act(z, "gelu_tanh")[2] - bo.act(z, "gelu")[2]) < 1e-3


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(8, 8), (7, 4), (6, 0)])
def test_norm_rope_gradients_are_differences(interleaved, D, rot):
    rng = np.random.default_rng(2)
    x, gamma = rng.standard_normal((2, 3, D)), rng.standard_normal(D)
    ang = rng.standard_normal((2, rot // 2))
    cos, sin = np.cos(ang), np.sin(ang)
    dy = rng.standard_normal((2, 3, D))
    loss = lambda: float((dy * bo.norm_rope(x, gamma, cos, sin, 1e-3, interleaved)).sum())  # noqa: E731
    dx, dgamma = bo.norm_rope_backward(dy, x, gamma, cos, sin, 1e-3, interleaved)
    assert np.abs(dx - difference(loss, x)).max() < 1e-7
    assert np.abs(dgamma - difference(loss, gamma)).max() < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_depends_on_distance(interleaved):
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    freq = 10.0 ** -np.arange(4)

    def at(x, p):
        a = (p * freq)[None]
        return bo.norm_rope(x, np.ones(8), np.cos(a), np.sin(a), 1e-12, interleaved)

    assert abs(np.linalg.norm(at(q, 5.0)) - math.sqrt(8)) < 1e-9
    one = float((at(q, 7.0) * at(k, 3.0)).sum())
    two = float((at(q, 11.0) * at(k, 7.0)).sum())
    assert abs(one - two) < 1e-12
    assert abs(one - float((at(q, 8.0) * at(k, 3.0)).sum())) > 1e-6


def test_clip_scales_to_the_norm():
    g = [np.array([3.0]), np.zeros(0), np.array([0.0, 4.0])]
    n, out = bo.clip(g, 1.0)
    assert n == 5.0 and abs(bo.grad_norm(out) - 1.0) < 1e-6
    n, out = bo.clip(g, 6.0)
    assert all(np.array_equal(a, b) for a, b in zip(out, g))
