"""The FP64 definitions of oracle/blocks.py against torch's autograd in FP64
and against identities that do not use their formulas."""
import numpy as np
import pytest
import torch

from oracle import blocks


@pytest.mark.parametrize("kind,f", [("silu", torch.nn.functional.silu),
                                    ("gelu", lambda a: torch.nn.functional.gelu(a, approximate="tanh"))])
def test_gated_and_its_gradients(kind, f):
    g = np.random.default_rng(1)
    x, w1, w3 = g.standard_normal((5, 8)), g.standard_normal((6, 8)), g.standard_normal((6, 8))
    a, u, h = blocks.gated(x, w1, w3, kind)
    ta, tu = torch.tensor(a, requires_grad=True), torch.tensor(u, requires_grad=True)
    th = f(ta) * tu
    assert np.allclose(h, th.detach().numpy(), rtol=1e-13, atol=1e-15)
    dh = g.standard_normal(h.shape)
    th.backward(torch.tensor(dh))
    d, again = blocks.gated_backward(dh, a, u, kind)
    assert np.array_equal(again, h)
    assert np.allclose(d, np.concatenate([ta.grad.numpy(), tu.grad.numpy()], axis=1), rtol=1e-12, atol=1e-14)


def test_logistic_far_out():
    v = np.array([-1e4, -745.0, 0.0, 40.0, 1e4, np.inf, -np.inf])
    z = blocks.logistic(v)
    assert z[0] == 0 and z[2] == 0.5 and z[4] == 1 and z[5] == 1 and z[6] == 0 and np.isfinite(z).all()


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("norm", [None, "rms", "layer"])
def test_heads_and_their_gradients(norm, adjacent):
    g = np.random.default_rng(2)
    T, H, D, rot = 4, 3, 10, 6
    x, w, dy = g.standard_normal((T, H, D)), 1 + 0.3 * g.standard_normal(D), g.standard_normal((T, H, D))
    freq, sections = np.array([1.0, 0.3, 0.01]), [2, 1]
    pos = g.integers(-50, 50, (T, 2))
    t = blocks.angles(pos, freq, sections)
    assert np.array_equal(t, np.stack([pos[:, 0] * 1.0, pos[:, 0] * 0.3, pos[:, 1] * 0.01], axis=1))
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    n = tx
    if norm == "rms":
        n = torch.nn.functional.rms_norm(tx, (D,), tw, 1e-6)
    if norm == "layer":
        n = torch.nn.functional.layer_norm(tx, (D,), tw, None, 1e-6)
    # the rotation as a product of complex numbers
    one, two = blocks.pairs(D, rot, adjacent)
    z = torch.complex(n[..., one], n[..., two]) * torch.polar(torch.ones(T, 1, 3, dtype=torch.float64),
                                                              torch.tensor(t)[:, None])
    y = n.clone()
    y[..., one], y[..., two] = z.real, z.imag
    W = None if norm is None else w
    assert np.allclose(blocks.head_norm_rotary(x, W, norm, 1e-6, t, adjacent), y.detach().numpy(), atol=1e-12)
    y.backward(torch.tensor(dy))
    dx, dw = blocks.head_norm_rotary_backward(dy, x, W, norm, 1e-6, t, adjacent)
    assert np.allclose(dx, tx.grad.numpy(), atol=1e-11)
    assert dw is None if norm is None else np.allclose(dw, tw.grad.numpy(), atol=1e-11)
