"""The centre network's operators in float64: linear layer, layer norm, their gradients, AdamW.

Written from the formulas, with no code in common with the library. Arrays are numpy float64.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 256          # elements of an 8-bit moment that share a scale
TOP = 448.0          # largest finite e4m3 value
TINY = 1e-30         # a block below this is stored as zeros

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def cdf(z):
    """The normal distribution function."""
    return 0.5 * _erfc(-np.asarray(z, dtype=np.float64) / math.sqrt(2.0))


def activation(z, act):
    if act in (None, "none"):
        return z
    if act == "tanh":
        return np.tanh(z)
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "gelu":
        return z * cdf(z)
    if act == "silu":
        return z / (1.0 + np.exp(-z))
    raise ValueError(act)


def activation_slope(z, act):
    if act in (None, "none"):
        return np.ones_like(z)
    if act == "tanh":
        return 1.0 - np.tanh(z) ** 2
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return cdf(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    raise ValueError(act)


def linear(x, w, b=None, act=None, residual=None):
    """(y, z): z = x w^T + b, y = act(z) + residual."""
    z = x @ w.T
    if b is not None:
        z = z + b
    y = activation(z, act)
    if residual is not None:
        y = y + residual
    return y, z


def linear_backward(g, x, w, z=None, act=None):
    """(grad_x, grad_w, grad_b, d) with d = g act'(z)."""
    d = g if act in (None, "none") else g * activation_slope(z, act)
    return d @ w, d.T @ x, d.sum(axis=0), d


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    mean = x.mean(axis=-1)
    c = x - mean[..., None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=-1) + eps)
    y = c * rstd[..., None]
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean, rstd


def layer_norm_backward(g, x, mean, rstd, w=None):
    h = (x - mean[..., None]) * rstd[..., None]
    t = g if w is None else g * w
    gx = rstd[..., None] * (t - t.mean(axis=-1, keepdims=True) - h * (t * h).mean(axis=-1, keepdims=True))
    axes = tuple(range(g.ndim - 1))
    return gx, (g * h).sum(axis=axes), g.sum(axis=axes)


def adamw(p, g, m, v, *, lr, beta1, beta2, eps, weight_decay, step, maximize=False):
    """(p, m, v) after one step; v is the second moment itself."""
    if maximize:
        g = -g
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    mh, vh = m / (1.0 - beta1 ** step), v / (1.0 - beta2 ** step)
    return p - lr * weight_decay * p - lr * mh / (np.sqrt(vh) + eps), m, v


def e4m3(x):
    """The nearest e4m3 value (ties to even), saturating at 448; steps of 2^-9 below 2^-6."""
    a = np.minimum(np.abs(x), TOP)
    _, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    return np.copysign(np.round(a / step) * step, x)


def pack(x, root=False):
    """(codes' values, scales) of a flat array: blocks of 256 in units of largest magnitude / 448;
    with ``root`` a positive value never becomes 0."""
    n = x.size
    blocks = -(-n // BLOCK)
    y = np.zeros(blocks * BLOCK)
    y[:n] = x
    y = y.reshape(blocks, BLOCK)
    top = np.abs(y).max(axis=1)
    scale = np.where(top < TINY, 0.0, top / TOP)
    safe = np.where(scale > 0, scale, 1.0)[:, None]
    q = np.where(scale[:, None] > 0, e4m3(y / safe), 0.0)
    if root:
        q = np.where((q == 0) & (y > 0) & (scale[:, None] > 0), 2.0 ** -9, q)
    return q.reshape(-1)[:n], scale


def unpack(q, scale):
    return q * np.repeat(scale, BLOCK)[:q.size]
