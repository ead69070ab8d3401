"""FP64 definitions of the layer operators: layer norm and its gradients, the
mixture-of-experts layer, adapters beside a quantized projection.

Written from the formulas, in numpy; no code is shared with the HIP library.
Inputs are float64 arrays of the exact input values (BF16 and FP32 values are
exact in float64); quantized operands are the oracle's codes and scales.
"""
from __future__ import annotations

import numpy as np

from . import e4m3
from . import quant

TILE = 128


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd) over the rows of x [R][C]."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, w=None):
    """(dx, dw, db) of sum(dy * y) for the given row statistics."""
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    c = x.shape[1]
    c1 = g.sum(axis=1, keepdims=True) / c
    c2 = (g * xhat).sum(axis=1, keepdims=True) / c
    return rstd[:, None] * (g - c1 - xhat * c2), (dy * xhat).sum(axis=0), dy.sum(axis=0)


def quant_tiles(y):
    """1x128 online quantization of float64 rows: codes uint8 [R][C], scales
    float32 [R][C/128], quotients float64 [R][C] (y / s, not yet rounded)."""
    y = np.asarray(y, np.float64)
    t = y.reshape(y.shape[0], -1, TILE)
    with np.errstate(invalid="ignore", divide="ignore"):
        amax = np.abs(t).max(axis=-1)
        s = quant.scale_from_amax(amax.astype(np.float32))
        quot = t / s[..., None].astype(np.float64)
    return e4m3.encode(quot).reshape(y.shape), s, quot.reshape(y.shape)


def code_spacing(quot):
    """Distance between the two E4M3 values around |quot| (<= 448)."""
    a = np.clip(np.abs(quot), 2.0 ** -6, 447.0)
    return 2.0 ** (np.floor(np.log2(a)) - 3)


def midpoint_distance(quot):
    """Distance of a quotient to the nearest rounding boundary of E4M3."""
    sp = code_spacing(quot)
    f = np.abs(quot) / sp
    return np.abs(f - np.floor(f) - 0.5) * sp


def route(logits, top_k, gate="softmax", bias=None, normalize=True, scale=1.0, ids=None):
    """(ids int [T][k] best first, gates [T][k]); equal values: lowest index.
    ids: a choice to take as given."""
    logits = np.asarray(logits, np.float64)
    if gate == "softmax":
        e = np.exp(logits - logits.max(axis=1, keepdims=True))
        score = e / e.sum(axis=1, keepdims=True)
    else:
        score = 1.0 / (1.0 + np.exp(-logits))
    value = logits if bias is None else score + bias
    if ids is None:
        ids = np.argsort(-value, axis=1, kind="stable")[:, :top_k]
    g = np.take_along_axis(score, ids, axis=1)
    if normalize:
        g = g / g.sum(axis=1, keepdims=True)
    return ids, g * scale


def moe(x_bits, router, w13, w2, top_k, first=0, **routing):
    """Whole layer in float64.  w13 / w2: lists (one per held expert) of
    (codes [2I][H], scales) and (codes [H][I], scales).  Returns y, ids, gates
    and, for tolerances, (magnitude, slack): sum |g| |W2| |h| per output, and
    what the outputs may move by because a quotient of h lies so near a
    rounding boundary that FP32 sums may put it on either side."""
    x = quant.bf16_to_f32(x_bits).astype(np.float64)
    T, H = x.shape
    ids, gates = route(x @ router.T, top_k, **routing)
    xq, xs = quant.quant_rows(x_bits)
    xd = quant.dequant_rows(xq, xs)
    y = np.zeros((T, H))
    mag, slack = np.zeros((T, H)), np.zeros((T, H))
    for j, ((q13, s13), (q2, s2)) in enumerate(zip(w13, w2)):
        rows, slot = np.nonzero(ids == first + j)
        if rows.size == 0:
            continue
        W13, W2 = quant.dequant_weight(q13, s13), quant.dequant_weight(q2, s2)
        inner = W2.shape[1]
        au = xd[rows] @ W13.T
        mau = np.abs(xd[rows]) @ np.abs(W13).T
        a, u = au[:, :inner], au[:, inner:]
        sil = a / (1.0 + np.exp(-a))
        h = sil * u
        # FP32 sums of n products and block folds: each of a, u within 2^-18
        # of its magnitude (fewer than 64 roundings); |silu'| <= 1.1
        dh = 2.0 ** -18 * (1.1 * mau[:, :inner] * np.abs(u) + np.abs(sil) * mau[:, inner:]) + 2.0 ** -20 * np.abs(h)
        q, s, quot = quant_tiles(h)
        sc = np.repeat(s.astype(np.float64), TILE, axis=1)
        tile_dh = np.repeat(dh.reshape(dh.shape[0], -1, TILE).max(axis=2), TILE, axis=1)
        near = midpoint_distance(quot) <= (dh + tile_dh * np.abs(quot) / 448.0) / sc
        hd = e4m3.decode(q) * sc
        g = gates[rows, slot][:, None]
        y[rows] += g * (hd @ W2.T)
        mag[rows] += np.abs(g) * (np.abs(hd) @ np.abs(W2).T)
        moved = near * code_spacing(quot) * sc + np.abs(hd) * (tile_dh / (448.0 * sc))
        slack[rows] += np.abs(g) * (moved @ np.abs(W2).T)
    return y, ids, gates, mag, slack


def adapters(x_bits, wq, ws, A, B, ids, scales=None):
    """Y in float64, and (sum |products| of the projection, of the adapters)."""
    x = quant.bf16_to_f32(x_bits).astype(np.float64)
    xq, xs = quant.quant_rows(x_bits)
    xd, W = quant.dequant_rows(xq, xs), quant.dequant_weight(wq, ws)
    y, mag = xd @ W.T, np.abs(xd) @ np.abs(W).T
    low = np.zeros_like(y)
    for a in range(A.shape[0]):
        rows = np.nonzero(ids == a)[0]
        if rows.size == 0:
            continue
        s = 1.0 if scales is None else float(scales[a])
        y[rows] += s * ((x[rows] @ A[a].T) @ B[a].T)
        low[rows] += abs(s) * ((np.abs(x[rows]) @ np.abs(A[a]).T) @ np.abs(B[a]).T)
    y[np.asarray(ids) >= A.shape[0]] = np.nan
    return y, mag, low
