"""The float64 oracle of the head's losses: its gradients against differences, and
values that are known without it."""

import numpy as np
import pytest

from oracle import loss_oracle as lo


def case(T=5, d=4, V=9, K=3, seed=0):
    rng = np.random.default_rng(seed)
    x, W = rng.standard_normal((T, d)), rng.standard_normal((V, d))
    idx = rng.integers(0, V, (T, K))
    idx[1, 2] = -1
    idx[2] = -1
    idx[3, 1] = idx[3, 0]  # the same index twice
    s = rng.standard_normal((T, K)) * 3
    s[0, 1] = -np.inf
    s[1, 2] = np.nan  # of no entry
    return x, W, idx, s, rng.uniform(0.1, 1, T)


@pytest.mark.parametrize("tau", [1.0, 2.0, 0.5])
@pytest.mark.parametrize("weighted", [False, True])
def test_gradients_are_the_differences(tau, weighted):
    x, W, idx, s, w = case()
    w = w if weighted else None
    _, _, dx, dW, _ = lo.head_loss(x, W, idx, s, w, tau)
    # central differences of step h are off by h^2 / 6 times the third derivative
    # (at most a few hundred here) and by 2^-52 |total| / h
    h, tol = 1e-5, 1e-7
    for a, g in ((x, dx), (W, dW)):
        for i in np.ndindex(a.shape):
            kept = a[i]
            a[i] = kept + h
            up = lo.head_loss(x, W, idx, s, w, tau)[1]
            a[i] = kept - h
            down = lo.head_loss(x, W, idx, s, w, tau)[1]
            a[i] = kept
            assert abs((up - down) / (2 * h) - g[i]) <= tol


def test_known_values():
    # equal logits: log V, whatever the target
    loss, total, dx, dW, _ = lo.cross_entropy(np.zeros((3, 2)), np.ones((8, 2)),
                                              np.array([1, -100, 7]), None)
    assert np.allclose(loss, [np.log(8), 0, np.log(8)]) and np.isclose(total, np.log(8))
    # the softmax's terms are rounded to 2^-53: eight times that at most
    assert np.abs(dx).max() <= 1e-15 and np.abs(dW).max() <= 1e-15
    # a student that agrees with its teacher over the whole vocabulary has no loss
    rng = np.random.default_rng(1)
    x, W = rng.standard_normal((4, 3)), rng.standard_normal((6, 3))
    idx = np.tile(np.arange(6), (4, 1))
    loss, _, dx, dW, _ = lo.head_loss(x, W, idx, x @ W.T + 5.0, None, 3.0)
    assert np.allclose(loss, 0) and np.allclose(dx, 0) and np.allclose(dW, 0)
    # one entry of a teacher is the cross entropy
    t = rng.integers(0, 6, 4)
    a = lo.head_loss(x, W, t[:, None], rng.standard_normal((4, 1)), None, 1.0)
    b = lo.cross_entropy(x, W, t, None)
    assert all(np.allclose(p, q) for p, q in zip(a[:4], b[:4]))


def test_no_token_counts():
    x, W, idx, s, w = case()
    loss, total, dx, dW, _ = lo.head_loss(x, W, np.full_like(idx, -1), s, w, 1.0)
    assert not loss.any() and total == 0 and not dx.any() and not dW.any()
