"""Measured cases of the operators between a layer's FP8 products: the gated
feed-forward product (both projections, activation and product), its backward
pass, and the norms of queries and keys with the position rotation, forward
and backward.

``run`` calls the package's operators where ``own`` is true; where it is false
it computes the same in elementary torch operations in FP32, rounded once at
the end.  ``exact`` computes the definitions in FP64.
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
E4M3_MAX = 448.0
SCALE_FLOOR = 1e-12
GELU_A, GELU_B = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def listed():
    return [
        # one decoded token through the wide gate and up projections
        dict(name="gated_token", op="gated", tokens=1, hidden=7168, inner=18432, act="silu", out="h"),
        # a decode batch at the expert's width, its codes for the down product
        dict(name="gated_decode", op="gated", tokens=48, hidden=7168, inner=2048, act="silu", out="codes"),
        # a training batch of an odd length: the projections are kept for the backward pass
        dict(name="gated_ragged", op="gated", tokens=1333, hidden=2048, inner=1408, act="gelu", out="kept"),
        # 4096 prompt tokens through the wide block: codes into the down product
        dict(name="gated_prompt", op="gated", tokens=4096, hidden=7168, inner=18432, act="silu", out="down"),
        # the backward pass of a small ragged batch, through to the gradients of x and of the weights
        dict(name="gated_train", op="gated_train", tokens=1333, hidden=2048, inner=1408, act="gelu"),
        # the backward pass of the wide block up to the operands of its products
        dict(name="gated_grad", op="gated_grad", tokens=4096, inner=18432, act="silu"),
        # one decoded token's heads, far into its sequence
        dict(name="heads_token", op="heads", tokens=1, q=32, k=8, dim=128, rot=128, x="bf16", w="bf16", norm="rms",
             adjacent=False, axes=1, start=100000),
        # a batch of prompts
        dict(name="heads_prompt", op="heads", tokens=8192, q=64, k=8, dim=128, rot=128, x="bf16", w="fp32", norm="rms",
             adjacent=False, axes=1, start=0),
        # patches of a video in FP32: three axes, a head size that fills no power of two
        dict(name="heads_video", op="heads", tokens=5003, q=16, k=16, dim=80, rot=80, x="fp32", w="fp32", norm="layer",
             adjacent=True, axes=3, start=0),
        # wide heads of which a part rotates, no norm, a decode batch far into its sequences
        dict(name="heads_partial", op="heads", tokens=64, q=128, k=1, dim=192, rot=64, x="bf16", w="bf16", norm="none",
             adjacent=True, axes=1, start=1000000),
        # the backward pass of a training batch
        dict(name="heads_grad", op="heads_grad", tokens=8192, q=32, k=8, dim=128, rot=128, x="bf16", w="fp32", norm="rms",
             adjacent=False, axes=1, start=0),
        # the same of the video's patches
        dict(name="heads_grad_video", op="heads_grad", tokens=5003, q=16, k=16, dim=80, rot=80, x="fp32", w="fp32",
             norm="layer", adjacent=True, axes=3, start=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_train", "gated_grad", "heads", "heads", "heads_grad"])
    act = rng.choice(["silu", "gelu"])
    if op == "gated":
        tokens = _log_int(rng, 1, 4096)
        return dict(op=op, tokens=tokens, hidden=128 * _log_int(rng, 4, 56), inner=128 * _log_int(rng, 1, 144), act=act,
                    out=rng.choice(["h", "kept", "codes" if tokens <= 64 else "down"]))
    if op == "gated_train":
        return dict(op=op, tokens=_log_int(rng, 1, 4096), hidden=128 * _log_int(rng, 4, 56),
                    inner=128 * _log_int(rng, 1, 56), act=act)
    if op == "gated_grad":
        return dict(op=op, tokens=_log_int(rng, 1, 4096), inner=128 * _log_int(rng, 1, 144), act=act)
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256, 2 * rng.randint(8, 128)])
    axes = rng.choice([1, 1, 2, 3])
    rot = rng.choice([dim, dim, dim // 4 * 2])
    q, k = _log_int(rng, 1, 64), _log_int(rng, 1, 16)
    tokens = _log_int(rng, 1, max(2, min(16384, 8192 * 36 * 128 // ((q + k) * dim))))
    return dict(op=op, tokens=tokens, q=q, k=k, dim=dim, rot=rot, x=rng.choice(["bf16", "bf16", "fp32"]),
                w=rng.choice(["bf16", "fp32"]), norm=rng.choice(["rms", "rms", "layer", "none"]),
                adjacent=rng.random() < 0.4, axes=axes, start=rng.choice([0, 0, _log_int(rng, 1, 1000000)]))


# ---------------------------------------------------------------- inputs

def _activations(g, rows, cols):
    """N(0, 1) with 16 outlier channels, as the quantizer's inputs have."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    ch = torch.randperm(cols, generator=g, device=DEV)[:16]
    boost = torch.where(torch.rand(rows, ch.numel(), generator=g, device=DEV) < 0.3, 20.0, 1.0)
    x[:, ch] = x[:, ch] * boost
    return x.bfloat16()


def _tiles_of(q):
    """Row-major codes [rows][cols] in the order of the GEMM's operand tiles."""
    rows, cols = q.shape
    # rows (r/16, r%16), columns (c/128, half of the 128, c/16 in the half, c%16)
    return q.view(rows // 16, 16, cols // 128, 2, 4, 16).permute(0, 2, 3, 4, 1, 5).reshape(rows, cols)


def _weight_codes(g, rows, cols, transposed=False):
    """Gaussian BF16 weights quantized in 128x128 blocks: operand-tiled E4M3
    codes and FP32 block scales [rows/128][cols/128]; transposed: the tiles
    of the transposed codes, which the input gradient reads."""
    w = (torch.randn(rows, cols, generator=g, device=DEV) * 0.02).bfloat16().float()
    b = w.view(rows // 128, 128, cols // 128, 128)
    s = (b.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp_min(SCALE_FLOOR)
    q = (b / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, cols)
    return _tiles_of(q.t().contiguous() if transposed else q), s


def _row_codes(x):
    """1x128 codes [T][K] and MN-major scales [K/128][T to a multiple of 4]."""
    q, s = _quant_rows(x.float())
    t = x.shape[0]
    pad = torch.zeros(s.shape[1], (t + 3) // 4 * 4, device=DEV)
    pad[:, :t] = s.t()
    return q.view(torch.uint8).view(x.shape), pad


def _positions(g, case):
    t, axes, start = case["tokens"], case["axes"], case["start"]
    i = torch.arange(t, device=DEV)
    if axes == 1:
        # prompts of up to 1000 tokens one behind the other, or tokens of sequences of various lengths
        if start:
            return start + torch.randint(0, start, (t,), generator=g, device=DEV)
        return i % 1000
    # a grid of patches, 24 x 16 a frame
    return torch.stack([i // 384, i // 16 % 24, i % 16][3 - axes:], dim=1) + start


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op == "gated":
        x = _activations(g, case["tokens"], case["hidden"])
        xq, xs = _row_codes(x)
        w13, s13 = _weight_codes(g, 2 * case["inner"], case["hidden"])
        s = dict(case=case, xq=xq, xs=xs, w13=w13, s13=s13)
        if case["out"] == "down":
            s["w2"], s["s2"] = _weight_codes(g, case["hidden"], case["inner"])
        return s
    if op in ("gated_train", "gated_grad"):
        t, i = case["tokens"], case["inner"]
        s = dict(case=case, dh=(1e-3 * torch.randn(t, i, generator=g, device=DEV)).bfloat16(),
                 gate_up=(1.5 * torch.randn(t, 2 * i, generator=g, device=DEV)).bfloat16())
        if op == "gated_train":
            s["x"] = _activations(g, t, case["hidden"])
            s["w13t"], s["s13"] = _weight_codes(g, 2 * i, case["hidden"], transposed=True)
        return s
    t, hq, hk, d, rot = case["tokens"], case["q"], case["k"], case["dim"], case["rot"]
    dt, wdt = _DT[case["x"]], _DT[case["w"]]
    # the projection's output: queries, keys and values of a token side by side
    s = dict(case=case, qkv=torch.randn(t, (hq + 2 * hk) * d, generator=g, device=DEV).mul_(2.0).to(dt),
             positions=_positions(g, case))
    if case["axes"] == 1:
        s["sections"] = None
        s["freq"] = 10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) / (rot // 2))
    else:
        n = rot // 2 // case["axes"]
        s["sections"] = [rot // 2 - n * (case["axes"] - 1)] + [n] * (case["axes"] - 1)
        s["freq"] = torch.cat([10000.0 ** (-torch.arange(m, device=DEV, dtype=torch.float64) / m) for m in s["sections"]])
    for n in ("wq", "wk"):
        s[n] = None if case["norm"] == "none" else (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(wdt)
    if op == "heads_grad":
        s["dq"] = (1e-3 * torch.randn(t, hq, d, generator=g, device=DEV)).to(dt)
        s["dk"] = (1e-3 * torch.randn(t, hk, d, generator=g, device=DEV)).to(dt)
    return s


def _heads(s):
    c = s["case"]
    t, hq, hk, d = c["tokens"], c["q"], c["k"], c["dim"]
    qkv = s["qkv"]
    return qkv[:, :hq * d].view(t, hq, d), qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)


# ---------------------------------------------------------------- plain form, FP32

def _untile(q):
    """Operand-tiled codes [rows][cols] -> their FP32 values, row-major."""
    rows, cols = q.shape
    v = q.view(torch.float8_e4m3fn).float().view(rows // 16, cols // 128, 2, 4, 16, 16)
    return v.permute(0, 4, 1, 2, 3, 5).reshape(rows, cols)


def _dequant_weight(q, s):
    rows, cols = q.shape
    return (_untile(q).view(rows // 128, 128, cols // 128, 128) * s[:, None, :, None]).view(rows, cols)


def _quant_rows(x):
    """1x128 tiles of FP32 rows: E4M3 codes, and the scales."""
    b = x.view(*x.shape[:-1], x.shape[-1] // 128, 128)
    amax = b.abs().amax(dim=-1)
    # a tensor of 448s: dividing by a number multiplies by its rounded inverse,
    # which moves the exact ties of BF16 rows
    s = (amax / torch.full_like(amax, E4M3_MAX)).clamp_min(SCALE_FLOOR)
    return (b / s[..., None]).to(torch.float8_e4m3fn), s


def _through_fp8(x):
    q, s = _quant_rows(x)
    return (q.float() * s[..., None]).view(x.shape)


def _columns(x):
    """x [T][C] as [C][T to a multiple of 128], zeros past the last token."""
    t, c = x.shape
    y = torch.zeros(c, (t + 127) // 128 * 128, device=x.device)
    y[:, :t] = x.t()
    return y


def _gate(a, act):
    """sigmoid's argument and its derivative."""
    if act == "silu":
        return a, torch.ones_like(a)
    return GELU_A * (a + GELU_B * a * a * a), GELU_A * (1.0 + 3.0 * GELU_B * a * a)


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _plain_gated(s):
    c = s["case"]
    t, k, i = c["tokens"], c["hidden"], c["inner"]
    x = s["xq"].view(torch.float8_e4m3fn).float().view(t, k // 128, 128) * s["xs"][:, :t].t()[:, :, None]
    au = x.view(t, k) @ _dequant_weight(s["w13"], s["s13"]).t()
    a, u = au[:, :i], au[:, i:]
    h = a * _sigmoid(_gate(a, c["act"])[0]) * u
    if c["out"] == "codes":
        q, sc = _quant_rows(h)
        return {"q": q.view(t, i), "s": sc.t().contiguous()}
    if c["out"] == "down":
        return {"y": (_through_fp8(h) @ _dequant_weight(s["w2"], s["s2"]).t()).bfloat16()}
    out = {"h": h.bfloat16()}
    if c["out"] == "kept":
        out["gate_up"] = au.bfloat16()
    return out


def _plain_gate_grads(s):
    """[da | du] in FP32."""
    c = s["case"]
    dh, au = s["dh"].float(), s["gate_up"].float()
    a, u = au[:, :c["inner"]], au[:, c["inner"]:]
    v, dv = _gate(a, c["act"])
    sig = _sigmoid(v)
    return torch.cat([dh * u * (sig + a * sig * (1.0 - sig) * dv), dh * (a * sig)], dim=1)


def _plain_gated_grad(s):
    d = _plain_gate_grads(s)
    q, sc = _quant_rows(d)
    dt = _columns(d)
    qt, st = _quant_rows(dt)
    return {"q": q.view(d.shape), "s": sc.t().contiguous(), "qt": qt.view(dt.shape), "st": st.t().contiguous()}


def _plain_gated_train(s):
    d = _plain_gate_grads(s)
    w13t = _untile(s["w13t"])
    rows, cols = w13t.shape
    w13t = (w13t.view(rows // 128, 128, cols // 128, 128) * s["s13"].t()[:, None, :, None]).view(rows, cols)
    dx = _through_fp8(d) @ w13t.t()
    dw = _through_fp8(_columns(d)) @ _through_fp8(_columns(s["x"].float())).t()
    return {"dx": dx.bfloat16(), "dw": dw.bfloat16()}


def _axis_of(s):
    """The position axis of each pair."""
    c = s["case"]
    axis = torch.zeros(c["rot"] // 2, dtype=torch.int64, device=DEV)
    if s["sections"] is not None:
        ends = torch.tensor(s["sections"], device=DEV).cumsum(0)
        axis = (torch.arange(c["rot"] // 2, device=DEV)[:, None] >= ends[None, :]).sum(dim=1)
    return axis


def _angles(s):
    """cos and sin [T][1][rot/2] of the angles, which take 64 bits far into a sequence."""
    p = s["positions"].view(s["case"]["tokens"], -1)[:, _axis_of(s)]
    a = p.double() * s["freq"]
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(x, cos, sin, case):
    rot = case["rot"]
    y = x.clone()
    if case["adjacent"]:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    else:
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return y


def _plain_norm(x, norm):
    """(normalized x, rstd)"""
    if norm == "none":
        return x, None
    if norm == "layer":
        x = x - x.mean(dim=-1, keepdim=True)
    rstd = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
    return x * rstd, rstd


def _plain_heads(s):
    c = s["case"]
    cos, sin = _angles(s)
    q, k = _heads(s)

    def one(x, w):
        n = _plain_norm(x.float(), c["norm"])[0]
        return _rotate(n if w is None else n * w.float(), cos, sin, c).to(x.dtype)

    return {"q": one(q, s["wq"]), "k": one(k, s["wk"])}


def _plain_heads_grad(s):
    c = s["case"]
    cos, sin = _angles(s)
    q, k = _heads(s)

    def one(dy, x, w):
        d = _rotate(dy.float(), cos, -sin, c)
        n, rstd = _plain_norm(x.float(), c["norm"])
        if rstd is None:
            return d.to(x.dtype), None
        g = d * w.float()
        dx = g - n * (g * n).mean(dim=-1, keepdim=True)
        if c["norm"] == "layer":
            dx = dx - g.mean(dim=-1, keepdim=True)
        return (rstd * dx).to(x.dtype), (d * n).sum(dim=(0, 1))

    dq, dwq = one(s["dq"], q, s["wq"])
    dk, dwk = one(s["dk"], k, s["wk"])
    out = {"dq": dq, "dk": dk}
    if dwq is not None:
        out.update(dwq=dwq, dwk=dwk)
    return out


_PLAIN = {"gated": _plain_gated, "gated_train": _plain_gated_train, "gated_grad": _plain_gated_grad,
          "heads": _plain_heads, "heads_grad": _plain_heads_grad}


def run(s):
    c = s["case"]
    if not own:
        return _PLAIN[c["op"]](s)
    import fine_grained_fp8_amd as fp8
    if c["op"] == "gated":
        if c["out"] in ("codes", "down"):
            q, sc = fp8.block_gemm_gated_quant(s["xq"], s["xs"], s["w13"], s["s13"], activation=c["act"])
            if c["out"] == "down":
                return {"y": fp8.block_gemm("fprop_tiled", q, sc, s["w2"], s["s2"])}
            return {"q": q.view(torch.float8_e4m3fn), "s": sc[:, :c["tokens"]]}
        if c["out"] == "h":
            return {"h": fp8.block_gemm_gated(s["xq"], s["xs"], s["w13"], s["s13"], activation=c["act"])}
        h, gate_up = fp8.block_gemm_gated(s["xq"], s["xs"], s["w13"], s["s13"], activation=c["act"], return_gate_up=True)
        return {"h": h, "gate_up": gate_up}
    if c["op"] == "gated_grad":
        q, sc, qt, st = fp8.gated_backward_quant(s["dh"], s["gate_up"], activation=c["act"])
        return {"q": q.view(torch.float8_e4m3fn), "s": sc[:, :c["tokens"]], "qt": qt.view(torch.float8_e4m3fn), "st": st}
    if c["op"] == "gated_train":
        q, sc, qt, st = fp8.gated_backward_quant(s["dh"], s["gate_up"], activation=c["act"])
        xt, xst = fp8.quant_act_cols(s["x"])
        return {"dx": fp8.block_gemm("dgrad_t_tiled", q, sc, s["w13t"], s["s13"]),
                "dw": fp8.block_gemm("wgrad_tiled", qt, st, xt, xst)}
    norm = None if c["norm"] == "none" else c["norm"]
    q, k = _heads(s)
    how = dict(q_weight=s["wq"], k_weight=s["wk"], norm=norm, eps=EPS, sections=s["sections"], adjacent=c["adjacent"])
    if c["op"] == "heads":
        q, k = fp8.head_norm_rotary(q, k, s["positions"], s["freq"], **how)
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = fp8.head_norm_rotary_backward(s["dq"], s["dk"], q, k, s["positions"], s["freq"], **how)
    return {"dq": dq, "dk": dk} if norm is None else {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, t = case["op"], case["tokens"]
    if op == "gated":
        k, i = case["hidden"], case["inner"]
        out = {"h": 2, "kept": 6, "codes": 1 + 1 / 32, "down": 0}[case["out"]] * t * i
        nbytes, flops = (t * k) * (1 + 1 / 32) + 2 * i * k + out, 4 * t * i * k + 8 * t * i
        if case["out"] == "down":
            return {"bytes": nbytes + i * k + 2 * t * k, "flops": flops + 2 * t * i * k}
        return {"bytes": nbytes, "flops": flops}
    if op == "gated_grad":
        n = t * case["inner"]
        return {"bytes": 6 * n + 4 * n * (1 + 1 / 32), "flops": 20 * n}
    if op == "gated_train":
        k, i = case["hidden"], case["inner"]
        return {"bytes": 6 * t * i + 2 * t * k + 2 * i * k + 2 * t * k + 4 * i * k, "flops": 8 * t * i * k + 20 * t * i}
    n = t * (case["q"] + case["k"]) * case["dim"]
    e = 2 if case["x"] == "bf16" else 4
    we = 2 if case["w"] == "bf16" else 4
    small = 8 * t * case["axes"] + 4 * case["rot"] + (0 if case["norm"] == "none" else 2 * we * case["dim"])
    if op == "heads":
        return {"bytes": 2 * e * n + small, "flops": 8 * n}
    return {"bytes": (3 if case["norm"] != "none" else 2) * e * n + small + 8 * case["dim"], "flops": 16 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def _values_of_codes(q):
    """E4M3 codes -> FP64, from the format: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    c = torch.arange(256, device=q.device)
    e, m = (c >> 3) & 15, (c & 7).double()
    f = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2(e.double() - 10.0))
    f = torch.where((c & 127) == 127, float("nan"), f)
    return torch.where(c >= 128, -f, f)[q.long()]


def _nearest_code_value(v):
    """The E4M3 value nearest to v (ties to the even mantissa, at most 448), in FP64."""
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -6)))
    e = torch.where(torch.pow(2.0, e) > a.clamp_min(2.0 ** -6), e - 1, e)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=v.device), e - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp_max(448.0)


def _tiles64(x):
    b = x.reshape(*x.shape[:-1], -1, 128)
    s = torch.clamp(b.abs().amax(dim=-1) / 448.0, min=1e-12).float().double()
    return _nearest_code_value((b / s[..., None]).float().double()), s


def _through64(x):
    q, s = _tiles64(x)
    return (q * s[..., None]).reshape(x.shape)


def _weights64(q, s):
    """FP64 weights [rows][cols] of one operand-tiled matrix; s [rows/128][cols/128]."""
    rows, cols = q.shape
    r = torch.arange(rows, device=q.device)[:, None]
    c = torch.arange(cols, device=q.device)[None, :]
    at = ((r // 16) * (cols // 128) + c // 128) * 2048 + ((c % 128) // 64) * 1024
    at = at + (((c % 64) // 16) * 16 + r % 16) * 16 + c % 16
    return _values_of_codes(q.reshape(-1)[at]) * s.double()[r // 128, c // 128]


def _act64(a, act):
    """act(a) and act'(a)"""
    if act == "silu":
        z = 1.0 / (1.0 + torch.exp(-a))
        return a * z, z * (1.0 + a * (1.0 - z))
    r = math.sqrt(2.0 / math.pi)
    th = torch.tanh(r * (a + GELU_B * a ** 3))
    return 0.5 * a * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * a * (1.0 - th * th) * r * (1.0 + 3.0 * GELU_B * a ** 2)


def _padded64(x):
    t = x.shape[0]
    return torch.cat([x, x.new_zeros((t + 127) // 128 * 128 - t, x.shape[1])]).t().contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    op, t = case["op"], case["tokens"]
    if op == "gated":
        k, i = case["hidden"], case["inner"]
        x = _values_of_codes(s["xq"]) * s["xs"][:, :t].double().t().repeat_interleave(128, dim=1)
        a = x @ _weights64(s["w13"][:i], s["s13"][:i // 128]).t()
        u = x @ _weights64(s["w13"][i:], s["s13"][i // 128:]).t()
        h = _act64(a, case["act"])[0] * u
        if case["out"] == "codes":
            q, sc = _tiles64(h)
            return {"q": q.reshape(t, i), "s": sc.t().contiguous()}
        if case["out"] == "down":
            return {"y": _through64(h) @ _weights64(s["w2"], s["s2"]).t()}
        return {"h": h, "gate_up": torch.cat([a, u], dim=1)} if case["out"] == "kept" else {"h": h}
    if op in ("gated_train", "gated_grad"):
        i = case["inner"]
        dh, a, u = s["dh"].double(), s["gate_up"][:, :i].double(), s["gate_up"][:, i:].double()
        f, df = _act64(a, case["act"])
        d = torch.cat([dh * u * df, dh * f], dim=1)
        if op == "gated_grad":
            q, sc = _tiles64(d)
            dt = _padded64(d)
            qt, st = _tiles64(dt)
            return {"q": q.reshape(d.shape), "s": sc.t().contiguous(), "qt": qt.reshape(dt.shape), "st": st.t().contiguous()}
        dx = _through64(d) @ _weights64(s["w13t"], s["s13"].t().contiguous()).t()
        return {"dx": dx, "dw": _through64(_padded64(d)) @ _through64(_padded64(s["x"].double())).t()}
    d, rot = case["dim"], case["rot"]
    sections = s["sections"] or [rot // 2]
    # the rotation of each token as a matrix on the head's channels
    pos = s["positions"].double().view(t, -1)
    angle, at = torch.zeros(t, rot // 2, dtype=torch.float64, device=DEV), 0
    for axis, n in enumerate(sections):
        angle[:, at:at + n] = pos[:, axis:axis + 1] * s["freq"][at:at + n]
        at += n
    j = torch.arange(rot // 2, device=DEV)
    first, second = (2 * j, 2 * j + 1) if case["adjacent"] else (j, j + rot // 2)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotated(v, by):
        z = torch.complex(v[..., first], v[..., second]) * by
        out = v.clone()
        out[..., first], out[..., second] = z.real.contiguous(), z.imag.contiguous()
        return out

    out = {}
    for name, x, w in zip("qk", _heads(s), (s["wq"], s["wk"])):
        x = x.double()
        mean = x.sum(-1, keepdim=True) / d if case["norm"] == "layer" else 0.0
        rstd = 1.0 if case["norm"] == "none" else (((x - mean) ** 2).sum(-1, keepdim=True) / d + EPS) ** -0.5
        xhat = (x - mean) * rstd
        w = torch.ones(d, dtype=torch.float64, device=DEV) if w is None else w.double()
        if op == "heads":
            out[name] = rotated(xhat * w, turn)
            continue
        dn = rotated(s["d" + name].double(), turn.conj())
        g = dn * w
        if case["norm"] == "none":
            out["d" + name] = g
            continue
        c1 = g.sum(-1, keepdim=True) / d if case["norm"] == "layer" else 0.0
        out["d" + name] = rstd * (g - c1 - xhat * ((g * xhat).sum(-1, keepdim=True) / d))
        out["dw" + name] = (dn * xhat).sum(0).sum(0)
    return out
