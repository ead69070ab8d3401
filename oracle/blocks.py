"""FP64 definitions of the operators between a layer's FP8 products: the gated
feed-forward product and its backward pass, head norms with the position
rotation and their backward pass.

Written from the formulas, in numpy; no code is shared with the HIP library.
Inputs are float64 arrays of the exact input values.
"""
from __future__ import annotations

import numpy as np


def logistic(v):
    v = np.asarray(v, np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def activation(a, kind):
    """act(a), its derivative, and (z, v, slope): act(a) = a z, z = logistic(v),
    slope = dv/da."""
    if kind == "silu":
        v, slope = a, np.ones_like(a)
    elif kind == "gelu":
        c = np.sqrt(2.0 / np.pi)
        v, slope = 2 * c * (a + 0.044715 * a ** 3), 2 * c * (1 + 3 * 0.044715 * a ** 2)
    else:
        raise ValueError(kind)
    z = logistic(v)
    return a * z, z + a * z * (1 - z) * slope, (z, v, slope)


def gated(x, w1, w3, kind="silu"):
    """(a, u, h) for x [M][K], w1 and w3 [I][K]."""
    a, u = x @ w1.T, x @ w3.T
    return a, u, activation(a, kind)[0] * u


def gated_backward(dh, a, u, kind="silu"):
    """([da | du], h)"""
    f, df, _ = activation(a, kind)
    return np.concatenate([dh * u * df, dh * f], axis=1), f * u


def angles(positions, freq, sections=None):
    """[T][pairs] from positions [T] or [T][axes]."""
    p = np.asarray(positions, np.float64).reshape(len(positions), -1)
    axis = np.zeros(len(freq), int) if sections is None else np.repeat(np.arange(len(sections)), sections)
    return p[:, axis] * np.asarray(freq, np.float64)


def pairs(dim, rot, adjacent):
    """First and second channel of the rotated pairs."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)


def rotate(n, t, adjacent):
    """n [T][H][D] with its first 2 * t.shape[1] channels rotated by the angles t [T][pairs]."""
    one, two = pairs(n.shape[2], 2 * t.shape[1], adjacent)
    y = n.copy()
    c, s = np.cos(t)[:, None], np.sin(t)[:, None]
    y[..., one] = n[..., one] * c - n[..., two] * s
    y[..., two] = n[..., two] * c + n[..., one] * s
    return y


def normalize(x, norm, eps):
    """(xhat, rstd [T][H][1])"""
    if norm is None:
        return x, np.ones(x.shape[:2] + (1,))
    d = x - x.mean(axis=2, keepdims=True) if norm == "layer" else x
    rstd = 1.0 / np.sqrt((d ** 2).mean(axis=2, keepdims=True) + eps)
    return d * rstd, rstd


def head_norm_rotary(x, w, norm, eps, t, adjacent):
    """x [T][H][D], w [D] or None, t [T][pairs]."""
    n = normalize(x, norm, eps)[0]
    return rotate(n if w is None else n * w, t, adjacent)


def head_norm_rotary_backward(dy, x, w, norm, eps, t, adjacent):
    """(dx, dw): dw as if a weight of ones were there where w is None."""
    d = rotate(dy, -t, adjacent)
    if norm is None:
        return d, None
    xhat, rstd = normalize(x, norm, eps)
    g = d if w is None else d * w
    dx = g - xhat * (g * xhat).mean(axis=2, keepdims=True)
    if norm == "layer":
        dx = dx - g.mean(axis=2, keepdims=True)
    return rstd * dx, (d * xhat).sum(axis=(0, 1))
