"""Float64 numpy definitions of the feed-forward operators and of gradient clipping: direct
formulas, no blocking, sharing no code with the CUDA path."""

from __future__ import annotations

import math

import numpy as np

ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    w = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
    return 0.5 * z * (1.0 + np.tanh(w))


def act_grad(z, name):
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    if name == "gelu":
        pdf = np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * pdf
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)


def linear(x, w, bias=None, residual=None, activation="none"):
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act(z, activation)
    return y if residual is None else y + residual


def linear_backward(x, w, bias, dy, activation="none"):
    z = x @ w.T
    if bias is not None:
        z = z + bias
    dz = dy * act_grad(z, activation)
    return dz @ w, dz.T @ x, dz.sum(0)


def gated(x, wg, wu, activation="silu"):
    return act(x @ wg.T, activation) * (x @ wu.T)


def gated_backward(x, wg, wu, dh, activation="silu"):
    g, u = x @ wg.T, x @ wu.T
    dg = dh * u * act_grad(g, activation)
    du = dh * act(g, activation)
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x


def grad_norm(grads, norm="l2"):
    if norm == "inf":
        return max((float(np.max(np.abs(g))) for g in grads if g.size), default=0.0)
    return math.sqrt(sum(float(np.sum(np.square(g))) for g in grads))


def clip(grads, max_norm, norm="l2"):
    total = grad_norm(grads, norm)
    c = min(1.0, max_norm / (total + 1e-6))
    return total, [g * c for g in grads]
