"""The operators between a layer's FP8 products on the GPU against their FP64
definitions (oracle/blocks.py).

Tolerances, all derived from the arithmetic (u = 2^-24; rounding to the output
type is off by at most half a step, eps / 2 of the value):
 - a and u of the gated product with exact products (up to 16 tokens, and up to 64
   where FP32 values or codes leave): at most 128 additions a K block in FP32,
   K / 128 folds of two roundings, a few merges of partial sums:
   (140 + 2 K / 128) u of the sum of magnitudes.
 - otherwise the FP8 MFMA truncates each product at 2^-13 of the largest of its
   group of 8 (test_gpu_accumulation.py), so a group loses at most 8 * 2^-13 of
   its largest, 2^-10 of its magnitudes; and the FP32 sums on top.
 - logistic: the exponential and the reciprocal 2^-22 of it, and an error e of its
   argument moves it by z (1 - z) e (GELU's argument: 4 roundings).
 - a head's sums pass 16 additions in a lane and at most 6 across lanes.
 - cos and sin: within 4 u.
"""
import numpy as np
import pytest
import torch

import synthetic as syn
from oracle import blocks, e4m3, layers, quant, tiling
from test_gpu_layers import codes_match, dev, host, rand, tile_codes

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------- the gated product

def activation_errors(a, ea, kind):
    """act(a), and bounds of its and its slope's errors for an a within ea."""
    f, df, (z, v, slope) = blocks.activation(a, kind)
    ez = z * (2.0 ** -22 + (1 - z) * (4 * U * np.abs(v) if kind == "gelu" else 0))
    ef = np.abs(a) * ez + U * np.abs(f)
    es = (np.abs(slope) if kind == "gelu" else 0) * 4 * U
    edf = ez + (ef * (1 - z) + np.abs(f) * (ez + U)) * np.abs(slope) + np.abs(f) * (1 - z) * es + 3 * U * (z + np.abs(f * (1 - z) * slope))
    # |act'| <= 1.13, |act''| <= 0.8 for both kinds
    return f, ef + 1.13 * ea + 0.4 * ea ** 2, df, edf + 0.8 * ea


class Gated:
    """A case's operands on both sides and what the definition says."""

    def __init__(self, M, K, I, kind, seed=1, std=0.05):
        self.kind, self.M, self.I = kind, M, I
        self.xq, self.xs = quant.quant_rows(syn.activation_with_outliers(M, K, seed=seed))
        self.wq, self.ws = quant.quant_weight(syn.gaussian((2 * I, K), seed=seed + 1, std=std))
        pad = np.zeros((K // 128, (M + 3) // 4 * 4), np.float32)
        pad[:, :M] = self.xs.T
        self.args = dev(self.xq), dev(pad), dev(tile_codes(self.wq)), dev(self.ws)
        self.K = K

    def define(self, dtype=torch.float32):
        x, w = quant.dequant_rows(self.xq, self.xs), quant.dequant_weight(self.wq, self.ws)
        au = x @ w.T
        mag = np.abs(x) @ np.abs(w).T
        few = (140 + 2 * self.K / 128) * U
        exact = self.M <= 16 or (self.M <= 64 and dtype == torch.float32)
        e = mag * (few if exact else few + 2.0 ** -10)
        i = self.I
        a, u = au[:, :i], au[:, i:]
        f, ef, _, _ = activation_errors(a, e[:, :i], self.kind)
        h = f * u
        return au, e, h, ef * (np.abs(u) + e[:, i:]) + np.abs(f) * e[:, i:] + 2 * U * np.abs(h)


def check(got, want, err, dtype, what):
    got = host(got)
    tol = err + (half_step(dtype)) * (np.abs(want) + err)
    bad = np.abs(got - want) / np.maximum(tol, 1e-300)
    assert (bad <= 1).all(), (what, float(bad.max()))


def normwise(got, want, dtype):
    # against the best answer of the type: the products' 1e-3 (both factors)
    best = torch.from_numpy(want).to(dtype).double().numpy()
    assert np.linalg.norm(host(got) - best) <= 2e-3 * np.linalg.norm(best)


def codes_of_f32(h):
    """Codes and scales [M][I/128] of FP32 values by the rule (R of the header)."""
    t = h.reshape(h.shape[0], -1, 128)
    s = quant.scale_from_amax(np.abs(t).max(axis=2))
    return e4m3.encode((t / s[..., None]).astype(np.float32)).reshape(h.shape), s


GATED = [  # M, K, I, kind
    (1, 128, 128, "silu"), (1, 1024, 384, "gelu"), (2, 256, 1408, "silu"), (15, 384, 256, "gelu"), (16, 128, 2048, "silu"),
    (17, 2048, 128, "silu"), (31, 640, 512, "gelu"), (33, 256, 4224, "silu"), (48, 1024, 256, "silu"), (49, 512, 8320, "gelu"),
    (64, 128, 384, "silu"), (64, 896, 2176, "gelu"), (5, 16384, 128, "silu"), (33, 4096, 256, "gelu"), (40, 384, 16384, "silu"),
    (65, 4096, 128, "gelu"), (200, 8192, 256, "silu"), (1000, 256, 1920, "gelu"), (65, 128, 128, "silu"), (90, 256, 16384, "silu"), (100, 384, 256, "gelu"), (128, 512, 128, "silu"), (129, 1024, 384, "silu"), (300, 640, 1408, "gelu"),
    (1333, 256, 512, "silu"), (700, 2560, 512, "gelu"), (333, 2944, 256, "silu"),
    (700, 256, 2048, "gelu"), (33, 256, 18432, "silu"), (60, 128, 24576, "gelu"),
    (1, 512, 9216, "silu"), (16, 384, 18432, "gelu"), (5, 128, 24576, "silu"), (9, 256, 8192, "gelu"),
    (450, 256, 4608, "silu"), (129, 384, 11264, "gelu"), (2300, 640, 1408, "gelu"), (1111, 128, 3840, "silu"),
]


@pytest.mark.parametrize("case", GATED, ids=lambda c: "-".join(map(str, c)))
def test_block_gemm_gated(gpu_lib, case):
    g = Gated(*case)
    for dtype in (torch.bfloat16, torch.float32):
        au, e, h, eh = g.define(dtype)
        y, kept = gpu_lib.block_gemm_gated(*g.args, activation=g.kind, out_dtype=dtype, return_gate_up=True)
        assert y.dtype == dtype and kept.dtype == torch.bfloat16
        check(y, h, eh, dtype, "h")
        normwise(y, h, dtype)
        check(kept, au, e, torch.bfloat16, "gate_up")
        assert torch.equal(y, gpu_lib.block_gemm_gated(*g.args, activation=g.kind, out_dtype=dtype))
    # the codes are those of the FP32 result
    q, s, again = gpu_lib.block_gemm_gated_quant(*g.args, activation=g.kind, return_gate_up=True)
    assert torch.equal(again, kept) and s.shape == (g.I // 128, (g.M + 3) // 4 * 4)
    qw, sw = codes_of_f32(y.cpu().numpy())
    assert np.array_equal(s[:, :g.M].t().cpu().numpy(), sw)
    assert np.array_equal(q.cpu().numpy(), qw)
    if g.M <= 64:
        codes_match(q, s, h, eh)
    q2, s2 = gpu_lib.block_gemm_gated_quant(*g.args, activation=g.kind)
    assert torch.equal(q, q2) and torch.equal(s[:, :g.M], s2[:, :g.M])


def test_gated_split_tail_and_wide_few(gpu_lib):
    """352 tiles (96 of them cut along K on 256 CUs), and a few tokens at a wide output."""
    for M, K, I in ((2700, 1024, 2048), (2100, 1024, 2048), (700, 1024, 2560), (3, 7168, 2048), (20, 1024, 18432), (7, 1024, 18432)):
        g = Gated(M, K, I, "silu", seed=5)
        rows = np.unique(np.concatenate([np.arange(0, M, 97), [M - 1]]))
        y = gpu_lib.block_gemm_gated(*g.args, out_dtype=torch.float32)
        q, s = gpu_lib.block_gemm_gated_quant(*g.args)
        qw, sw = codes_of_f32(y.cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), qw) and np.array_equal(s[:, :M].t().cpu().numpy(), sw)
        part = Gated.__new__(Gated)
        part.__dict__.update(g.__dict__, xq=g.xq[rows], xs=g.xs[rows])
        _, _, h, eh = part.define()
        check(y[torch.from_numpy(rows).cuda()], h, eh, torch.float32, (M, K, I))
        assert torch.equal(y, gpu_lib.block_gemm_gated(*g.args, out_dtype=torch.float32))


def test_gated_equals_the_plain_products(gpu_lib):
    """More than 64 tokens: a and u are the block GEMM's own sums."""
    for M, I in ((200, 384), (450, 4608)):
        g = Gated(M, 512, I, "silu", seed=9)
        A, sA, w, sw = g.args
        _, kept = gpu_lib.block_gemm_gated(A, sA, w, sw, return_gate_up=True)
        assert torch.equal(kept, gpu_lib.block_gemm("fprop_tiled", A, sA, w, sw))


@pytest.mark.parametrize("M,I", [(9, 384), (50, 384), (150, 384), (450, 4608)])
def test_gated_strides_and_rows_behind(gpu_lib, M, I):
    """Operands and outputs inside larger arrays: nothing else is written."""
    K = 256
    g = Gated(M, K, I, "silu", seed=11)
    A, sA, w, sw = g.args
    bigA = torch.full((M + 3, K + 48), 0x7F, dtype=torch.uint8, device="cuda")
    bigA[:M, 16:16 + K] = A
    big_s = torch.full((K // 128, sA.shape[1] + 5), float("nan"), device="cuda")
    big_s[:, :sA.shape[1]] = sA
    big_w = torch.full((2 * I // 128, K // 128 + 3), float("nan"), device="cuda")
    big_w[:, :K // 128] = sw
    out = torch.full((M + 2, I + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    y = gpu_lib.block_gemm_gated(bigA[:M, 16:16 + K], big_s[:, :M], w, big_w[:, :K // 128], out=out[:M, 8:8 + I])
    want = gpu_lib.block_gemm_gated(A, sA, w, sw)
    assert torch.equal(y, want)
    assert (out[M:] == 7).all() and (out[:, :8] == 7).all() and (out[:, 8 + I:] == 7).all()


@pytest.mark.parametrize("M,I", [(5, 256), (40, 256), (130, 256), (450, 4608)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_nonfinite_tokens_stay_apart(gpu_lib, M, I, kind):
    g = Gated(M, 256, I, kind, seed=13)
    A, sA, w, sw = g.args
    clean = gpu_lib.block_gemm_gated(A, sA, w, sw, activation=kind)
    qc, sc = gpu_lib.block_gemm_gated_quant(A, sA, w, sw, activation=kind)
    A, sA = A.clone(), sA.clone()
    A[1, 3] = 0x7F
    sA[0, M - 1] = float("inf")
    y = gpu_lib.block_gemm_gated(A, sA, w, sw, activation=kind)
    q, s = gpu_lib.block_gemm_gated_quant(A, sA, w, sw, activation=kind)
    keep = [i for i in range(M) if i not in (1, M - 1)]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(q[keep], qc[keep]) and torch.equal(s[:, keep], sc[:, keep])
    assert y[1].isnan().all() and (q[1] == 0x7F).all() and s[:, 1].isnan().all()
    assert not y[M - 1].isfinite().any() and not s[:, M - 1].isfinite().any()


def test_gated_far_gates(gpu_lib):
    """Gates far on both sides: act(a) is a, or vanishes without a NaN."""
    K = 128
    for M in (4, 100, 42000):
        A = torch.full((M, K), 0x7E, dtype=torch.uint8, device="cuda")        # 448
        sA = torch.ones(1, (M + 3) // 4 * 4, device="cuda")
        w = np.full((512, K), 0x7E, np.uint8)
        w[:128] = 0xFE                                                        # gates at -448^2 128 s
        sw = torch.ones(4, 1, device="cuda")
        for scale in (1.0, 1e-5, 1e30):
            y = gpu_lib.block_gemm_gated(A, sA, dev(tile_codes(w)), sw * scale, out_dtype=torch.float32)
            a = 448.0 * 448.0 * 128 * float(np.float32(scale))
            f = blocks.activation(np.array([-a, a]), "silu")[0]
            want = np.float32(f * a)       # an overflow is infinite in FP32
            assert np.allclose(y[0, [0, 200]].cpu().numpy(), want, rtol=1e-6, atol=1e-30)


def test_gated_empty(gpu_lib):
    A = torch.empty(0, 256, dtype=torch.uint8, device="cuda")
    w, sw = torch.zeros(512, 256, dtype=torch.uint8, device="cuda"), torch.ones(4, 2, device="cuda")
    y, kept = gpu_lib.block_gemm_gated(A, torch.empty(2, 0, device="cuda"), w, sw, return_gate_up=True)
    assert y.shape == (0, 256) and kept.shape == (0, 512)


@pytest.mark.parametrize("I", [8320, 18432])
def test_gated_empty_and_wide(gpu_lib, I):
    """No tokens, more channels than the kernel for few of them takes."""
    A, sA = torch.empty(0, 128, dtype=torch.uint8, device="cuda"), torch.empty(1, 0, device="cuda")
    w, sw = torch.zeros(2 * I, 128, dtype=torch.uint8, device="cuda"), torch.ones(2 * I // 128, 1, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        y, kept = gpu_lib.block_gemm_gated(A, sA, w, sw, out_dtype=dtype, return_gate_up=True)
        assert y.shape == (0, I) and y.dtype == dtype and kept.shape == (0, 2 * I)
    q, s, kept = gpu_lib.block_gemm_gated_quant(A, sA, w, sw, return_gate_up=True)
    assert q.shape == (0, I) and s.shape == (I // 128, 0) and kept.shape == (0, 2 * I)


# ------------------------------------------------------------- its backward pass

def backward_errors(dh, a, u, kind):
    f, ef, df, edf = activation_errors(a, 0.0, kind)
    d, h = blocks.gated_backward(dh, a, u, kind)
    e = np.concatenate([np.abs(dh * u) * edf + 3 * U * np.abs(dh * u * df), np.abs(dh) * ef + 2 * U * np.abs(dh * f)], axis=1)
    return d, e, h, ef * np.abs(u) + 2 * U * np.abs(h)


def padded_t(a):
    out = np.zeros((a.shape[1], (a.shape[0] + 127) // 128 * 128))
    out[:, :a.shape[0]] = a.T
    return out


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("T,I", [(1, 128), (3, 256), (127, 128), (128, 384), (129, 128), (300, 640), (1000, 1408), (1501, 1408)])
def test_gated_backward(gpu_lib, T, I, kind):
    dh, gu = rand((T, I), 21, torch.bfloat16, std=1e-3), rand((T, 2 * I), 22, torch.bfloat16, std=2.0)
    gu[0, 0], gu[0, 1], gu[0, 2] = -30.0, 60.0, 0.0
    D, A, B = host(dh), host(gu[:, :I]), host(gu[:, I:])
    d, e, h, eh = backward_errors(D, A, B, kind)
    check(gpu_lib.gated_backward(dh, gu, activation=kind), d, e, torch.bfloat16, "d")
    q, s, qt, st, ht, sht = gpu_lib.gated_backward_quant(dh, gu, activation=kind, return_h=True)
    codes_match(q, s, d, e)
    codes_match(qt, st, padded_t(d), padded_t(e))
    ht_rows = torch.from_numpy(tiling.untile_codes(ht.cpu().numpy(), I, ht.shape[1]))
    codes_match(ht_rows, sht, padded_t(h), padded_t(eh))
    without = gpu_lib.gated_backward_quant(dh, gu, activation=kind)
    assert torch.equal(q, without[0]) and torch.equal(s[:, :T], without[1][:, :T])
    assert torch.equal(qt, without[2]) and torch.equal(st, without[3])


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_backward_of_far_gates(gpu_lib, kind):
    """act'(a) is 1 or vanishes, without a NaN, up to the largest finite gates."""
    far = torch.tensor([200.0, 1e10, 4e19, 1e20, 1e30, 3e38], dtype=torch.bfloat16, device="cuda")
    for T in (2, 16500):                    # a set of values and all of them to a workgroup
        dh = torch.full((T, 128), 2.0 ** -4, dtype=torch.bfloat16, device="cuda")
        gu = torch.full((T, 256), 2.0, dtype=torch.bfloat16, device="cuda")
        gu[:, :6], gu[:, 6:12] = far, -far
        d = gpu_lib.gated_backward(dh, gu, activation=kind)
        q, s, _, _, ht, sht = gpu_lib.gated_backward_quant(dh, gu, activation=kind, return_h=True)
        assert d.isfinite().all() and s[:, :T].isfinite().all()
        assert (d[:, :6] == 2.0 ** -3).all() and (d[:, 6:12] == 0).all()
        assert torch.equal(d[:, 128:134], (far.float() * 2.0 ** -4).bfloat16().expand(T, 6)) and (d[:, 134:140] == 0).all()
        assert ((q[:, 6:12] & 0x7F) == 0).all() and not ((q & 0x7F) == 0x7F).any()


def test_gated_backward_against_differences(gpu_lib):
    g = np.random.default_rng(3)
    bf = lambda x: torch.from_numpy(x).bfloat16()
    a, u, dh = (bf(g.standard_normal((4, 128))) for _ in range(3))
    for kind in ("silu", "gelu"):
        d = host(gpu_lib.gated_backward(dh.cuda(), torch.cat([a, u], 1).cuda(), activation=kind))
        A, B, D = (t.double().numpy() for t in (a, u, dh))
        f = lambda A_, B_: D * blocks.activation(A_, kind)[0] * B_
        t = 1e-6
        da, du = (f(A + t, B) - f(A - t, B)) / (2 * t), (f(A, B + t) - f(A, B - t)) / (2 * t)
        want = np.concatenate([da, du], 1)
        # truncation t^2, FP64 rounding 1e-16 / t, and the result's own rounding
        assert (np.abs(d - want) <= half_step(torch.bfloat16) * np.abs(want) + 1e-8).all()


@pytest.mark.parametrize("T", [150, 8300])       # a set of values and all of them to a workgroup
def test_gated_backward_strides_nonfinite_and_zero(gpu_lib, T):
    I = 256
    big_dh, big_gu = rand((T + 1, I + 8), 31, torch.bfloat16), rand((T + 1, 2 * I + 24), 32, torch.bfloat16)
    dh, gu = big_dh[:T, 8:], big_gu[:T, 16:16 + 2 * I]
    want = gpu_lib.gated_backward_quant(dh.contiguous(), gu.contiguous(), return_h=True)
    got = gpu_lib.gated_backward_quant(dh, gu, return_h=True)
    for i, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x[:, :T], y[:, :T]) if i == 1 else torch.equal(x, y)
    dh, gu = dh.contiguous(), gu.contiguous()
    dh[5, 7] = float("nan")
    dh[140, 200] = float("inf")
    dh[:, 128:] *= 0
    dh[140, 200] = float("inf")
    gu[140, 200], gu[140, I + 200] = 1.0, 1.0
    q, s, qt, st, _, _ = gpu_lib.gated_backward_quant(dh, gu, return_h=True)
    q, s, qt, st = (t.cpu().numpy() for t in (q, s, qt, st))
    for half in (0, I):                     # da and du
        assert np.isnan(s[half // 128, 5]) and (q[5, half:half + 128] == 0x7F).all()
        assert np.isnan(st[0, half + 7]) and (qt[half + 7, :128] == 0x7F).all() and np.isfinite(st[1, half + 7])
        assert np.isinf(s[half // 128 + 1, 140]) and q[140, half + 200] == 0x7F
        assert ((np.delete(q[140, half + 128:half + 256], 72) & 0x7F) == 0).all()
        assert np.isinf(st[1, half + 200]) and qt[half + 200, 140] == 0x7F
        assert ((np.delete(qt[half + 200, 128:], 12) & 0x7F) == 0).all()
        assert (s[half // 128 + 1, :140] == np.float32(1e-12)).all() and (st[0, half + 128:half + 256] == np.float32(1e-12)).all()


@pytest.mark.parametrize("rows,cols", [(1, 128), (127, 256), (128, 128), (130, 384), (1333, 1024)])
def test_quant_act_cols(gpu_lib, rows, cols):
    bits = syn.activation_with_outliers(rows, cols, seed=41)
    pad = np.zeros(((rows + 127) // 128 * 128, cols), np.uint16)
    pad[:rows] = bits
    qw, sw = quant.quant_cols(pad)
    big = torch.full((rows + 1, cols + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:rows, :cols] = dev(bits.view(np.int16)).view(torch.bfloat16)
    q, s = gpu_lib.quant_act_cols(big[:rows, :cols])
    assert np.array_equal(tiling.untile_codes(q.cpu().numpy(), cols, pad.shape[0]), qw)
    assert np.array_equal(s.t().cpu().numpy(), sw)


def test_the_dense_example_and_its_gradients(gpu_lib):
    """Norm, projection, heads and feed-forward block as the example joins them, ragged
    tokens, against the unquantized computation in FP64 and its gradients there."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decoder_block as ex
    torch.manual_seed(3)
    T, H = 333, 256
    b = ex.Dense(H, 384, heads=8, kv_heads=2, dim=64)
    b.q_weight += 0.3 * torch.randn(64, device="cuda")
    b.k_weight += 0.3 * torch.randn(64, device="cuda")
    x = rand((T, H), 61, torch.bfloat16)
    dq, dk, dv = (rand((T, h, 64), 62 + h, torch.bfloat16, std=0.1) for h in (8, 2, 2))
    dy = rand((T, H), 66, torch.bfloat16, std=0.1)
    pos = torch.arange(T, device="cuda") + 5000
    outs, grads = ex.dense_step(b, x, pos, dq, dk, dv, dy)

    leaf = lambda t: t.detach().double().cpu().requires_grad_()
    n = leaf(torch.nn.functional.layer_norm(x.double(), (H,), eps=1e-5))
    w = {k: leaf(v) for k, v in b.weights.items()}
    qw, kw = leaf(b.q_weight), leaf(b.k_weight)
    t = (n @ w["qkv"].T).view(T, 12, 64)
    turn = pos.cpu().double()[:, None, None] * b.freq.cpu()
    c, s = turn.cos(), turn.sin()

    def rotated(h, weight):
        h = h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight
        return torch.cat([h[..., :32] * c - h[..., 32:] * s, h[..., 32:] * c + h[..., :32] * s], -1)
    gu = n @ w["w13"].T
    want = rotated(t[:, :8], qw), rotated(t[:, 8:10], kw), t[:, 10:], torch.nn.functional.silu(gu[:, :384]) * gu[:, 384:] @ w["w2"].T
    torch.autograd.backward(want, [g.double().cpu() for g in (dq, dk, dv, dy)])
    # E4M3 rounds each operand by at most 2^-4; two to four quantized products follow each other
    bound = 4 * 2.0 ** -4
    names = dict(n=n, **w, q_weight=qw, k_weight=kw)
    for got, ref in [*zip(outs, want), *((grads[k], v.grad) for k, v in names.items())]:
        ref = ref.detach().numpy()
        assert np.linalg.norm(host(got) - ref) <= bound * np.linalg.norm(ref)


def test_a_whole_feed_forward_block_and_its_gradients(gpu_lib):
    """x -> codes -> gated product -> down product, and back, ragged tokens: the
    operators together, on the codes that they hand to each other."""
    T, K, I = 333, 256, 384
    x = rand((T, K), 51, torch.bfloat16)
    w13 = rand((2 * I, K), 52, torch.bfloat16, std=0.08)
    w2 = rand((K, I), 53, torch.bfloat16, std=0.08)
    dy = rand((T, K), 54, torch.bfloat16, std=1e-2)
    q13, s13, q13t = gpu_lib.quant_weight_128x128(w13, transposed=True, tiled=True)
    q2, s2, q2t = gpu_lib.quant_weight_128x128(w2, transposed=True, tiled=True)
    xq, xs, _ = gpu_lib.quant_act_1x128(x)
    hq, hs, kept = gpu_lib.block_gemm_gated_quant(xq, xs, q13, s13, return_gate_up=True)
    y = gpu_lib.block_gemm("fprop_tiled", hq, hs, q2, s2)
    dyq, dys, _ = gpu_lib.quant_act_1x128(dy)
    dh = gpu_lib.block_gemm("dgrad_t_tiled", dyq, dys, q2t, s2)
    q, s, qt, st, ht, sht = gpu_lib.gated_backward_quant(dh, kept, return_h=True)
    dx = gpu_lib.block_gemm("dgrad_t_tiled", q, s, q13t, s13)
    xt, xst = gpu_lib.quant_act_cols(x)
    dw13 = gpu_lib.block_gemm("wgrad_tiled", qt, st, xt, xst, out_dtype=torch.float32)
    dyp = torch.zeros(384, K, dtype=torch.bfloat16, device="cuda")
    dyp[:T] = dy
    dyt, dyst, _ = gpu_lib.quant_act_1x128(dyp, "col")
    dw2 = gpu_lib.block_gemm("wgrad_tiled", dyt, dyst, ht, sht, out_dtype=torch.float32)
    # against the unquantized block in FP64: E4M3 rounds each operand by at most 2^-4 (2.5%
    # by 2-norm for spread values), and two to four quantized products follow each other
    X, W13, W2, DY = host(x), host(w13), host(w2), host(dy)
    a, u, h = blocks.gated(X, W13[:I], W13[I:])
    DH = DY @ W2
    D, _ = blocks.gated_backward(DH, a, u)
    for got, want in ((y, h @ W2.T), (dx, D @ W13), (dw13, D.T @ X), (dw2, DY.T @ h)):
        assert np.linalg.norm(host(got) - want) <= 4 * 2.0 ** -4 * np.linalg.norm(want)


# ------------------------------------------------------------- heads

def head_case(T, H, D, dtype, seed, stride="fused"):
    """x [T][H][D] as a view with the stride asked for."""
    if stride == "fused":      # heads of a wider row, 16-byte aligned
        return rand((T, (H + 2) * D), seed, dtype, mean=0.2)[:, D:(H + 1) * D].view(T, H, D)
    if stride == "odd":        # no row starts aligned
        return rand((T, H * (D + 1) + 3), seed, dtype, mean=0.2)[:, 1:1 + H * (D + 1)].view(T, H, D + 1)[:, :, :D]
    return rand((H, T, D), seed, dtype, mean=0.2).transpose(0, 1)      # head by head


def head_bounds(x, w, norm, eps, t, adjacent):
    """What n (before the rotation) may be off by, and each value's partner's size."""
    xhat, rstd = blocks.normalize(x, norm, eps)
    W = 1.0 if w is None else np.abs(w)
    n = np.abs(xhat) * W
    en = np.zeros_like(n) if norm is None else 32 * U * n
    if norm == "layer":
        dm = 26 * U * np.abs(x).mean(axis=2, keepdims=True) * rstd        # the mean, in units of xhat
        en = en + W * (dm + np.abs(xhat) * (0.5 * dm ** 2 + dm * np.abs(xhat.mean(axis=2, keepdims=True))))
    return n, en


def with_partner(v, pairs_, ):
    one, two = pairs_
    out = v.copy()
    out[..., one] += v[..., two]
    out[..., two] += v[..., one]
    return out


def head_tolerance(x, w, norm, eps, t, adjacent):
    n, en = head_bounds(x, w, norm, eps, t, adjacent)
    p = blocks.pairs(x.shape[2], 2 * t.shape[1], adjacent)
    turned = np.zeros(x.shape[2], bool)
    turned[p[0]] = turned[p[1]] = True
    return with_partner(en, p) + turned * 6 * U * with_partner(n, p)


HEADS = [  # T, Hq, Hk, D, rot, norm, adjacent, sections, stride
    (1, 1, 0, 128, 128, "rms", False, None, "fused"),
    (1, 32, 8, 128, 128, "rms", False, None, "fused"),
    (7, 5, 1, 64, 64, "rms", True, None, "fused"),
    (5, 3, 2, 80, 80, "layer", True, [14, 13, 13], "fused"),
    (9, 4, 4, 96, 32, None, True, None, "fused"),
    (6, 9, 2, 192, 64, "rms", False, [20, 6, 6], "fused"),
    (3, 2, 1, 256, 256, "layer", False, [64, 32, 16, 16], "heads"),
    (4, 2, 1, 512, 512, "rms", False, None, "fused"),
    (2, 3, 1, 1024, 1024, "rms", True, None, "fused"),
    (5, 3, 2, 72, 40, "rms", False, None, "odd"),
    (4, 2, 2, 2, 2, "layer", True, None, "odd"),
    (3, 5, 1, 130, 66, "layer", False, [33, 0], "odd"),
    (3, 1, 1, 1022, 1022, "rms", False, None, "odd"),
    (3, 2, 0, 128, 0, "rms", False, None, "heads"),
    (2, 0, 3, 16, 16, "rms", False, None, "fused"),
    (300, 16, 2, 128, 64, "rms", False, None, "heads"),
    (5000, 3, 1, 64, 64, "layer", False, None, "fused"),
]


def head_inputs(case, x_dtype, w_dtype, seed=61):
    T, Hq, Hk, D, rot, norm, adjacent, sections, stride = case
    q = head_case(T, Hq, D, DT[x_dtype], seed, stride) if Hq else None
    k = head_case(T, Hk, D, DT[x_dtype], seed + 1, stride) if Hk else None
    wq = rand(D, seed + 2, DT[w_dtype], mean=1.0, std=0.3) if norm and Hq else None
    wk = rand(D, seed + 3, DT[w_dtype], mean=1.0, std=0.3) if norm and Hk else None
    g = np.random.default_rng(seed)
    freq = 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    pos = g.integers(-1000, 1000000, (T,) if sections is None else (T, len(sections)))
    t = blocks.angles(pos, freq, sections) if rot else np.zeros((T, 0))
    rotary = (torch.from_numpy(pos).cuda().to(torch.int32 if T % 2 else torch.int64), dev(freq)) if rot else (None, None)
    how = dict(q_weight=wq, k_weight=wk, norm=norm, eps=1e-6, sections=sections, adjacent=adjacent)
    return q, k, rotary, how, t


@pytest.mark.parametrize("x_dtype,w_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("case", HEADS, ids=lambda c: "-".join(str(v).replace(" ", "") for v in c))
def test_head_norm_rotary(gpu_lib, case, x_dtype, w_dtype):
    q, k, rotary, how, t = head_inputs(case, x_dtype, w_dtype)
    out = gpu_lib.head_norm_rotary(q, k, *rotary, **how)
    for x, y, w in ((q, out[0], how["q_weight"]), (k, out[1], how["k_weight"])):
        if x is None:
            assert y is None
            continue
        assert y.dtype == x.dtype and y.shape == x.shape
        X, W = host(x), None if w is None else host(w)
        want = blocks.head_norm_rotary(X, W, how["norm"], how["eps"], t, how["adjacent"])
        check(y, want, head_tolerance(X, W, how["norm"], how["eps"], t, how["adjacent"]), x.dtype, case)
        if how["norm"] is None:          # channels that do not rotate are copied
            assert torch.equal(y[..., 2 * t.shape[1]:], x[..., 2 * t.shape[1]:])


@pytest.mark.parametrize("x_dtype,w_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("case", HEADS, ids=lambda c: "-".join(str(v).replace(" ", "") for v in c))
def test_head_norm_rotary_backward(gpu_lib, case, x_dtype, w_dtype):
    q, k, rotary, how, t = head_inputs(case, x_dtype, w_dtype)
    stride = case[-1]
    dq, dk = (None if x is None else head_case(*x.shape, x.dtype, 71 + i, stride) for i, x in enumerate((q, k)))
    out = gpu_lib.head_norm_rotary_backward(dq, dk, q, k, *rotary, **how)
    norm, adjacent = how["norm"], how["adjacent"]
    for i, (x, dy, w) in enumerate(((q, dq, how["q_weight"]), (k, dk, how["k_weight"]))):
        dx, dw = out[i], out[2 + i]
        if x is None:
            assert dx is None and dw is None
            continue
        assert dx.dtype == x.dtype and dx.shape == x.shape
        X, DY, W = host(x), host(dy), None if w is None else host(w)
        want, want_w = blocks.head_norm_rotary_backward(DY, X, W, norm, how["eps"], t, adjacent)
        p = blocks.pairs(X.shape[2], 2 * t.shape[1], adjacent)
        m = with_partner(np.abs(DY), p)                  # what d's terms add up to
        if norm is None:
            check(dx, want, 6 * U * m, x.dtype, case)
            assert dw is None
            continue
        xhat, rstd = blocks.normalize(X, norm, how["eps"])
        xh = np.abs(xhat)
        dxh = (26 * U * np.abs(X).mean(axis=2, keepdims=True) * rstd if norm == "layer" else 0) * np.ones_like(xh)
        gm = m * (1.0 if W is None else np.abs(W))
        mean = lambda v: v.mean(axis=2, keepdims=True)
        e = rstd * (128 * U * (gm + mean(gm) + xh * mean(gm * xh)) + dxh * mean(gm * xh) + xh * mean(gm * dxh) + dxh * mean(gm * dxh))
        check(dx, want, e, x.dtype, case)
        n = X.shape[0] * X.shape[1] + 64
        assert dw.dtype == torch.float32
        assert (np.abs(host(dw) - want_w) <= (n * U * m * xh + m * dxh).sum(axis=(0, 1)) + 1e-30).all()
    again = gpu_lib.head_norm_rotary_backward(dq, dk, q, k, *rotary, **how)
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("norm", [None, "rms", "layer"])
def test_head_gradients_against_differences(gpu_lib, norm):
    T, H, D, rot = 3, 2, 16, 12
    x, dy = rand((T, H, D), 81, torch.float32), rand((T, H, D), 82, torch.float32)
    w = None if norm is None else rand(D, 83, torch.float32, mean=1.0)
    freq, pos = 2.0 ** -np.arange(rot // 2), np.array([-7, 0, 100])
    t = blocks.angles(pos, freq)
    dx, _, dw, _ = gpu_lib.head_norm_rotary_backward(dy, None, x, None, dev(pos), dev(freq), q_weight=w, norm=norm, eps=1e-3)
    X, D_, W = host(x), host(dy), None if w is None else host(w)
    loss = lambda X_, W_: (D_ * blocks.head_norm_rotary(X_, W_, norm, 1e-3, t, False)).sum(axis=2)
    s = 1e-5
    for c in range(D):
        e = np.zeros(D)
        e[c] = s
        # truncation s^2 times third derivatives of order 10, FP64 rounding 1e-16 / s, FP32 results
        assert np.allclose((loss(X + e, W) - loss(X - e, W)) / (2 * s), host(dx)[..., c], atol=2e-5, rtol=2e-5)
        if w is not None:
            assert np.isclose((loss(X, W + e) - loss(X, W - e)).sum() / (2 * s), host(dw)[c], atol=5e-5, rtol=2e-5)


def test_heads_into_one_row_and_nothing_else(gpu_lib):
    """Queries and keys of a fused projection, in and out, forward and backward."""
    T, Hq, Hk, D = 37, 6, 2, 64
    for dtype in (torch.bfloat16, torch.float32):
        qkv = rand((T, (Hq + 2 * Hk) * D), 91, dtype)
        q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        out = torch.full((T + 1, (Hq + 2 * Hk) * D), 7.0, dtype=dtype, device="cuda")
        oq, ok = out[:T, :Hq * D].view(T, Hq, D), out[:T, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        rotary = torch.arange(T, device="cuda"), dev(0.9 ** np.arange(32))
        want = gpu_lib.head_norm_rotary(q, k, *rotary)
        gpu_lib.head_norm_rotary(q, k, *rotary, out=(oq, ok))
        assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])
        assert (out[T:] == 7).all() and (out[:, (Hq + Hk) * D:] == 7).all()
        dq, dk, wq, wk = gpu_lib.head_norm_rotary_backward(*want, q, k, *rotary)
        out.fill_(7.0)
        _, _, wq2, wk2 = gpu_lib.head_norm_rotary_backward(*want, q, k, *rotary, out=(oq, ok))
        assert torch.equal(oq, dq) and torch.equal(ok, dk) and torch.equal(wq, wq2) and torch.equal(wk, wk2)
        assert (out[T:] == 7).all() and (out[:, (Hq + Hk) * D:] == 7).all()


@pytest.mark.parametrize("what", ["weight", "one_token", "one_head"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_aligned_heads_whatever_is_not_read_in_pieces(gpu_lib, dtype, what):
    """A weight that starts anywhere, and strides that no step is taken along, change
    nothing: the same sums in the same order, bit for bit."""
    dtype = DT[dtype]
    T, Hq, Hk, D = {"weight": (40, 6, 2, 128), "one_token": (1, 6, 2, 128), "one_head": (40, 1, 1, 128)}[what]
    rotary = torch.arange(T, device="cuda") + 9, dev(0.9 ** np.arange(D // 2))
    w = rand(2 * D + 2, 141, dtype, mean=1.0, std=0.3)
    w = w[1:1 + D], w[D + 1:2 * D + 1]
    heads = [rand((T, h, D), 142 + i, dtype) for i, h in enumerate((Hq, Hk, Hq, Hk))]
    plain = [v.clone() for v in w]
    want = gpu_lib.head_norm_rotary(*heads[:2], *rotary, q_weight=plain[0], k_weight=plain[1])
    want_grad = gpu_lib.head_norm_rotary_backward(heads[2], heads[3], *heads[:2], *rotary, q_weight=plain[0], k_weight=plain[1])
    if what != "weight":
        w = plain
        odd = (lambda t: t.as_strided(t.shape, (t.numel() + 3, D, 1))) if what == "one_token" else \
            (lambda t: t.as_strided(t.shape, (D, D + 3, 1)))
        heads = [odd(t) for t in heads]
    else:
        assert all(v.data_ptr() % 16 for v in w)
    out = [torch.empty_like(t) for t in heads]
    got = gpu_lib.head_norm_rotary(*heads[:2], *rotary, q_weight=w[0], k_weight=w[1], out=(out[0], out[1]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = gpu_lib.head_norm_rotary_backward(heads[2], heads[3], *heads[:2], *rotary, q_weight=w[0], k_weight=w[1], out=(out[2], out[3]))
    assert all(torch.equal(a, b) for a, b in zip(got, want_grad))


def test_heads_nonfinite_values_stay_apart(gpu_lib):
    T, H, D, rot = 4, 3, 64, 32
    x = rand((T, H, D), 95, torch.float32)
    rotary = torch.arange(T, device="cuda"), dev(0.9 ** np.arange(rot // 2))
    for norm in (None, "rms", "layer"):
        clean = gpu_lib.head_norm_rotary(x, None, *rotary, norm=norm)[0]
        y = x.clone()
        y[1, 2, 40] = float("nan")       # a channel that does not rotate
        y[2, 0, 63] = float("inf")
        got = gpu_lib.head_norm_rotary(y, None, *rotary, norm=norm)[0]
        touched = torch.zeros(T, H, D, dtype=torch.bool, device="cuda")
        if norm is None:
            touched[1, 2, 40] = touched[2, 0, 63] = True
        else:
            touched[1, 2] = touched[2, 0] = True
        assert torch.equal(got[~touched], clean[~touched])
        assert got[1, 2, 40].isnan() and (norm is not None or got[2, 0, 63] == float("inf"))


def test_heads_constant_and_zero(gpu_lib):
    x = torch.zeros(3, 2, 128, device="cuda")
    x[1] = 3.0
    y = gpu_lib.head_norm_rotary(x, None, norm="layer")[0]
    assert (y == 0).all()
    y = gpu_lib.head_norm_rotary(x, None, norm="rms")[0]
    assert (y[0] == 0).all() and torch.allclose(y[1], torch.ones_like(y[1]), rtol=1e-6)


def test_heads_empty(gpu_lib):
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    rotary = torch.empty(0, dtype=torch.int64, device="cuda"), dev(0.9 ** np.arange(32))
    assert gpu_lib.head_norm_rotary(q, None, *rotary)[0].shape == (0, 4, 64)
    dq, dk, wq, wk = gpu_lib.head_norm_rotary_backward(q, None, q, None, *rotary)
    assert dq.shape == (0, 4, 64) and dk is None and wk is None and (wq == 0).all()


def test_a_set_without_heads(gpu_lib):
    """It has results without heads and a gradient of zeros; the other set is as alone."""
    T = 300
    none = torch.empty(T, 0, 64, device="cuda")
    k, dk = rand((T, 3, 64), 91, torch.float32), rand((T, 3, 64), 92, torch.float32)
    w = rand((64,), 93, torch.float32)
    rotary = torch.arange(T, device="cuda"), dev(0.9 ** np.arange(32))
    y, yk = gpu_lib.head_norm_rotary(none, k, *rotary, q_weight=w, k_weight=w)
    assert y.shape == (T, 0, 64) and torch.equal(yk, gpu_lib.head_norm_rotary(None, k, *rotary, k_weight=w)[1])
    alone = gpu_lib.head_norm_rotary_backward(None, dk, None, k, *rotary, k_weight=w)
    torch.full((4096,), float("nan"), device="cuda")           # what the next allocation holds
    dq, dx, dwq, dwk = gpu_lib.head_norm_rotary_backward(none, dk, none, k, *rotary, q_weight=w, k_weight=w)
    assert dq.shape == (T, 0, 64) and dwq.shape == (64,) and (dwq == 0).all()
    assert torch.equal(dx, alone[1]) and torch.equal(dwk, alone[3])


def test_rows_past_32_bit_offsets(gpu_lib):
    """Heads and gates whose elements lie more than 2^31 (2^32 bytes) into their arrays."""
    T, H, D = 70000, 256, 128                     # 2.3e9 elements
    x = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 10000):
        x[i:i + 10000].normal_()
    rotary = torch.arange(T, device="cuda"), dev(10000.0 ** (-np.arange(64) / 64))
    y = gpu_lib.head_norm_rotary(x, None, *rotary)[0]
    last = gpu_lib.head_norm_rotary(x[-9:].contiguous(), None, rotary[0][-9:].contiguous(), rotary[1])[0]
    assert torch.equal(y[-9:], last)
    dx = gpu_lib.head_norm_rotary_backward(y, None, x, None, *rotary)[0]
    last = gpu_lib.head_norm_rotary_backward(y[-9:].contiguous(), None, x[-9:].contiguous(), None, rotary[0][-9:].contiguous(), rotary[1])[0]
    assert torch.equal(dx[-9:], last)
    del y, dx
    I = 16384
    flat = x.view(-1)
    dh, gu = flat[:65600 * I].view(-1, I), flat[:65600 * 2 * I].view(-1, 2 * I)    # 2.1e9 elements of gate_up
    d = gpu_lib.gated_backward(dh, gu)
    tail = gpu_lib.gated_backward(dh[-64:].contiguous(), gu[-64:].contiguous())
    assert torch.equal(d[-64:], tail)


# ------------------------------------------------------------- streams, graphs, refusals

def block_calls(gpu_lib, seed=101):
    """Every operator at a few-token and a larger size: (inputs that change, call)."""
    calls = []
    for M in (12, 200):
        g = Gated(M, 384, 256, "silu", seed=seed)
        A, sA, w, sw = g.args
        calls.append(([A], lambda A, sA=sA, w=w, sw=sw: gpu_lib.block_gemm_gated(A, sA, w, sw, return_gate_up=True)))
        calls.append(([A], lambda A, sA=sA, w=w, sw=sw: gpu_lib.block_gemm_gated_quant(A, sA, w, sw)[:1]))
        dh, gu = rand((M, 256), seed + 1, torch.bfloat16), rand((M, 512), seed + 2, torch.bfloat16)
        calls.append(([dh, gu], lambda dh, gu: [t for i, t in enumerate(gpu_lib.gated_backward_quant(dh, gu, return_h=True)) if i != 1]))
        calls.append(([dh], lambda dh: gpu_lib.quant_act_cols(dh)))
        q, k = rand((M, 8, 128), seed + 3, torch.bfloat16), rand((M, 2, 128), seed + 4, torch.bfloat16)
        pos, freq = torch.arange(M, device="cuda") + 5, dev(10000.0 ** (-np.arange(64) / 64))
        calls.append(([q, k, pos], lambda q, k, pos, freq=freq: gpu_lib.head_norm_rotary(q, k, pos, freq)))
        dq, dk = rand((M, 8, 128), seed + 5, torch.bfloat16), rand((M, 2, 128), seed + 6, torch.bfloat16)
        calls.append(([dq, dk, q, pos], lambda dq, dk, q, pos, k=k, freq=freq:
                      gpu_lib.head_norm_rotary_backward(dq, dk, q, k, pos, freq)))
    A, sA, w, sw = Gated(450, 256, 4608, "silu", seed=seed).args           # the block GEMM's kernel
    calls.append(([A], lambda A: gpu_lib.block_gemm_gated(A, sA, w, sw, return_gate_up=True)))
    return calls


def test_blocks_replay_from_graphs(gpu_lib):
    """Each operator captured; replayed several times with other inputs and eager work of
    its own between, always equal to the eager result."""
    calls = block_calls(gpu_lib)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for ins, call in calls:
            call(*ins)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [call(*ins) for ins, call in calls]
    for turn in range(4):
        for ins, _ in calls:
            for t in ins:
                t.copy_(t.roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        held = [[t.clone() for t in out] for out in outs]
        for (ins, call), got in zip(calls, held):
            want = call(*ins)
            for a, b in zip(got, want):
                assert torch.equal(a, b), turn
        torch.cuda.synchronize()


def test_two_graphs_of_the_gated_product_at_once(gpu_lib):
    """Two captures of a product whose tail is cut along K when it runs eagerly,
    replayed on two streams at once."""
    g = [Gated(2700, 512, 2048, "silu", seed=s) for s in (111, 112)]
    want = [gpu_lib.block_gemm_gated(*x.args, out_dtype=torch.float32) for x in g]
    graphs, outs = [], []
    for x in g:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(gpu_lib.block_gemm_gated(*x.args, out_dtype=torch.float32))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, gr in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            # other places for the cuts of K: FP32 sums in another order
            assert torch.allclose(o, w, rtol=1e-4, atol=1e-4 * float(w.abs().max()))
    first = [o.clone() for o in outs]
    for gr in graphs:
        gr.replay()
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))


def test_blocks_on_other_streams(gpu_lib):
    """Two streams at once, tensors made on the current one; results as on that."""
    calls = block_calls(gpu_lib, 121)
    want = [call(*ins) for ins, call in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for n, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for ins, call in calls:
                outs[n].append(call(*ins))
    torch.cuda.synchronize()
    for out in outs:
        for got, ref in zip(out, want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
    s = streams[0]
    q = rand((33, 4, 64), 131, torch.bfloat16)
    s.wait_stream(torch.cuda.current_stream())
    y = gpu_lib.head_norm_rotary(q, None, stream=s)[0]
    s.synchronize()
    assert torch.equal(y, gpu_lib.head_norm_rotary(q, None)[0])


def test_block_refusals(gpu_lib):
    A, s, w = torch.zeros(4, 256, dtype=torch.uint8, device="cuda"), torch.ones(2, 4, device="cuda"), \
        torch.zeros(512, 256, dtype=torch.uint8, device="cuda")
    sw = torch.ones(4, 2, device="cuda")
    f = gpu_lib.block_gemm_gated
    assert f(A, s, w, sw).shape == (4, 256)
    for bad in (lambda: f(A, s, w[:384], sw), lambda: f(A, s[:1], w, sw), lambda: f(A, s, w, sw[:3]), lambda: f(A, s, w, sw, activation="relu"),
                lambda: f(A, s, w, sw, out=torch.empty(4, 128, device="cuda")), lambda: f(A.cpu(), s, w, sw), lambda: f(A, s, w.cpu(), sw)):
        with pytest.raises((ValueError, gpu_lib.FP8Error)):
            bad()
    for dtype in (torch.float16, torch.float64):
        with pytest.raises(TypeError):
            f(A, s, w, sw, out_dtype=dtype)
    dh, gu = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        gpu_lib.gated_backward(dh, gu[:, :128])
    with pytest.raises(gpu_lib.FP8Error):
        gpu_lib.gated_backward(dh[:, :64], gu[:, :128])
    with pytest.raises(TypeError):
        gpu_lib.gated_backward(dh.float(), gu)
    h = gpu_lib.head_norm_rotary
    q, pos, freq = torch.zeros(4, 2, 64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(32, dtype=torch.float64, device="cuda")
    assert h(q, None, pos, freq)[0].shape == q.shape
    for bad in (lambda: h(None, None), lambda: h(q, q[:3], pos, freq), lambda: h(q, q.bfloat16(), pos, freq), lambda: h(q, None, pos),
                lambda: h(q, None, pos.float(), freq), lambda: h(q, None, pos[:3], freq), lambda: h(q, None, pos, freq.float()),
                lambda: h(q, None, pos, torch.ones(33, dtype=torch.float64, device="cuda")), lambda: h(q, None, pos, freq, sections=[16, 16]),
                lambda: h(q, None, pos, freq, norm="l2"), lambda: h(q, None, pos, freq, norm=None, q_weight=torch.ones(64, device="cuda")),
                lambda: h(q, None, pos, freq, q_weight=torch.ones(63, device="cuda")), lambda: h(q.transpose(1, 2), None, pos, freq),
                lambda: h(q, None, pos, freq, out=(q, None)), lambda: h(q[:, :, :63], None), lambda: h(q.expand(4, 2, 64)[:, :1].expand(4, 5, 64), None),
                lambda: h(q.double(), None), lambda: h(q.cpu(), None), lambda: h(q, None, pos, freq, eps=-1.0)):
        with pytest.raises((ValueError, TypeError, gpu_lib.FP8Error)):
            bad()
    b = gpu_lib.head_norm_rotary_backward
    for bad in (lambda: b(q, None, None, None, pos, freq), lambda: b(q, None, q[:, :1], None, pos, freq), lambda: b(q, None, q.bfloat16(), None, pos, freq)):
        with pytest.raises((ValueError, TypeError)):
            bad()
