"""Float64 oracle of the operators around the projections: the matrix product
with bias, activation and residual, the norm of queries and keys with the
rotary embedding, and the clip of many gradients with Adam.  Plain numpy,
shares no code with the CUDA library."""

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])
C = math.sqrt(2.0 / math.pi)


def act(z, name):
    if name == "relu":
        return np.where(z > 0, z, 0.0 * z)
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(C * (z + 0.044715 * z ** 3)))
    return z


def act_grad(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    if name == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-z * z / 2) / math.sqrt(
            2 * math.pi)
    if name == "gelu_tanh":
        t = np.tanh(C * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C * (1 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def linear(x, W, bias, residual, name):
    """(y, z)"""
    z = x @ W.T
    if bias is not None:
        z = z + bias
    y = act(z, name)
    return (y if residual is None else y + residual), z


def linear_backward(dy, z, W, name):
    """(dx, dbias, dz)"""
    dz = dy * act_grad(z, name)
    return dz @ W, dz.sum(0), dz


def _pairs(rot, interleaved):
    h = rot // 2
    i = np.arange(h)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + h)


def norm_rope(x, gamma, cos, sin, eps, interleaved):
    """x [T][heads][D]; cos, sin [T][rot/2]: the rows of the tokens' positions."""
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * gamma
    a, b = _pairs(2 * cos.shape[1], interleaved)
    y = n.copy()
    c, s = cos[:, None, :], sin[:, None, :]
    y[..., a] = n[..., a] * c - n[..., b] * s
    y[..., b] = n[..., b] * c + n[..., a] * s
    return y


def norm_rope_backward(dy, x, gamma, cos, sin, eps, interleaved):
    """(dx, dgamma)"""
    a, b = _pairs(2 * cos.shape[1], interleaved)
    c, s = cos[:, None, :], sin[:, None, :]
    dn = dy.copy()
    dn[..., a] = dy[..., a] * c + dy[..., b] * s
    dn[..., b] = dy[..., b] * c - dy[..., a] * s
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    g = dn * gamma
    dx = r * (g - x * r * r * np.mean(g * x, -1, keepdims=True))
    return dx, (dn * x * r).sum((0, 1))


def grad_norm(grads):
    # scaled by the largest magnitude: squares of float64 can overflow too
    top = max((float(np.max(np.abs(g))) for g in grads if g.size), default=0.0)
    if top == 0.0 or not np.isfinite(top):
        return top
    return top * math.sqrt(sum(float(np.sum((g / top) ** 2)) for g in grads))


def clip(grads, max_norm):
    n = grad_norm(grads)
    scale = min(1.0, max_norm / (n + 1e-6))
    return n, [g * scale for g in grads]
