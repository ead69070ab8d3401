"""CPU pins of the FP64 definitions in oracle/layers.py: closed forms,
differences, and agreement with independent ways to compute the same."""
import numpy as np
import torch

import synthetic as syn
from oracle import e4m3, layers, quant


def test_layer_norm_closed_form_and_torch():
    y, mean, rstd = layers.layer_norm(np.array([[1.0, 3.0], [5.0, 5.0]]), eps=0.25)
    assert np.allclose(mean, [2, 5]) and np.allclose(rstd, [1 / np.sqrt(1.25), 2])
    assert np.allclose(y, [[-1 / np.sqrt(1.25), 1 / np.sqrt(1.25)], [0, 0]])
    g = np.random.default_rng(0)
    x, w, b = g.standard_normal((7, 33)), g.standard_normal(33), g.standard_normal(33)
    t = torch.nn.functional.layer_norm(torch.from_numpy(x), (33,), torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    assert np.allclose(layers.layer_norm(x, w, b)[0], t.numpy(), atol=1e-12)


def test_layer_norm_backward_against_differences():
    g = np.random.default_rng(1)
    x, dy, w, b = g.standard_normal((4, 9)), g.standard_normal((4, 9)), g.standard_normal(9), g.standard_normal(9)
    _, mean, rstd = layers.layer_norm(x, w, b)
    dx, dw, db = layers.layer_norm_backward(dy, x, mean, rstd, w)
    h = 1e-6
    for c in range(9):
        e = np.eye(9)[c] * h
        f = lambda x_, w_, b_: (dy * layers.layer_norm(x_, w_, b_)[0]).sum(axis=1)
        assert np.allclose((f(x + e, w, b) - f(x - e, w, b)) / (2 * h), dx[:, c], atol=1e-7)
        assert np.isclose((f(x, w + e, b) - f(x, w - e, b)).sum() / (2 * h), dw[c], atol=1e-7)
        assert np.isclose((f(x, w, b + e) - f(x, w, b - e)).sum() / (2 * h), db[c], atol=1e-7)


def test_quant_tiles_equals_the_row_quantizer_on_bf16_values():
    xb = syn.activation_with_outliers(16, 512, seed=2)
    q, s, quot = layers.quant_tiles(quant.bf16_to_f32(xb))
    qo, so = quant.quant_rows(xb)
    assert np.array_equal(s, so)
    same = q == qo
    # FP64 quotients are not rounded to FP32 first: they differ at boundaries alone,
    # by an FP32 rounding of a quotient of up to 448
    assert (layers.midpoint_distance(quot)[~same] <= 448 * 2.0 ** -24).all()
    assert np.array_equal(e4m3.encode(quot.astype(np.float32)), qo)
    assert (np.abs(e4m3.decode(q) - quot) <= layers.code_spacing(quot) / 2 + 1e-12).all()


def test_route_orders_ties_and_normalizes():
    l = np.array([[0.0, 2.0, 2.0, -1.0, 1.0]])
    ids, g = layers.route(l, 3)
    assert ids.tolist() == [[1, 2, 4]] and np.isclose(g.sum(), 1)
    ids, g = layers.route(l, 2, gate="sigmoid", bias=np.array([9, 0, 0, 0, 0.0]), normalize=False, scale=2.0)
    assert ids.tolist() == [[0, 1]] and np.allclose(g, [[1.0, 2 / (1 + np.exp(-2.0))]])


def test_moe_shares_add_up():
    T, H, I, E, k = 4, 128, 128, 4, 2
    xb, R = syn.gaussian((T, H), seed=3), np.random.default_rng(4).standard_normal((E, H)) * 0.1
    w13 = [quant.quant_weight(syn.gaussian((2 * I, H), seed=5 + e, std=0.05)) for e in range(E)]
    w2 = [quant.quant_weight(syn.gaussian((H, I), seed=15 + e, std=0.05)) for e in range(E)]
    whole = layers.moe(xb, R, w13, w2, k)[0]
    parts = sum(layers.moe(xb, R, w13[f:f + 2], w2[f:f + 2], k, f)[0] for f in (0, 2))
    assert np.allclose(whole, parts, rtol=1e-12)
    assert np.abs(whole).max() > 0


def test_adapters_equal_a_merged_weight():
    T, K, N, r, n = 6, 128, 128, 8, 2
    xb = syn.gaussian((T, K), seed=6)
    wq, ws = quant.quant_weight(syn.gaussian((N, K), seed=7, std=0.02))
    g = np.random.default_rng(8)
    A, B = g.standard_normal((n, r, K)), g.standard_normal((n, N, r))
    ids = np.array([0, 1, -1, 1, 0, 2])
    y, _, _ = layers.adapters(xb, wq, ws, A, B, ids, [0.5, 2.0])
    base, _, _ = layers.adapters(xb, wq, ws, A, B, np.full(T, -1))
    x = quant.bf16_to_f32(xb).astype(np.float64)
    assert np.allclose(y[0] - base[0], 0.5 * (B[0] @ A[0]) @ x[0])
    assert np.allclose(y[3] - base[3], 2.0 * (B[1] @ A[1]) @ x[3])
    assert np.array_equal(y[2], base[2]) and np.isnan(y[5]).all()
