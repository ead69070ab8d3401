"""Measured cases of the operators around the FP8 products: layer norm (forward,
with and without the fused 1x128 quantization, and backward), the whole
mixture-of-experts layer for a few tokens, and low-rank adapters beside a
shared FP8 projection.

``run`` calls the package's operators where ``own`` is true; where it is false
it computes the same in elementary torch operations in FP32, rounded once at
the end.  ``exact`` computes the definitions in FP64.
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5
E4M3_MAX = 448.0
SCALE_FLOOR = 1e-12


def listed():
    return [
        # one decoded token of the 7168-wide layer: latency of the norm alone
        dict(name="norm_token", op="norm", rows=1, cols=7168, x="bf16", w="fp32", quant=False),
        # a training or prompt batch of the quantizer's size, the norm feeding an FP8 product
        dict(name="norm_quant_batch", op="norm", rows=8192, cols=7168, x="bf16", w="bf16", quant=True),
        # an FP32 residual stream of an odd width: no row but the first is 16-byte aligned
        dict(name="norm_odd_fp32", op="norm", rows=3001, cols=2047, x="fp32", w="fp32", quant=False),
        # the backward pass of the training batch
        dict(name="norm_grad_batch", op="norm_grad", rows=8192, cols=7168, x="bf16", w="fp32"),
        # many short rows (a norm over the channels of one head), gradients in FP32
        dict(name="norm_grad_heads", op="norm_grad", rows=20011, cols=128, x="fp32", w="fp32"),
        # one decoded token through a layer of 8 experts, two of them chosen
        dict(name="experts_token", op="experts", tokens=1, hidden=7168, inner=2048, experts=8, first=0,
             local=8, top_k=2, gate="softmax", bias=False),
        # a decode batch on one GPU's share: 8 of 64 experts held here, biased sigmoid router
        dict(name="experts_share", op="experts", tokens=32, hidden=7168, inner=2048, experts=64, first=16,
             local=8, top_k=6, gate="sigmoid", bias=True),
        # the largest decode batch, many small experts, every expert held here
        dict(name="experts_batch", op="experts", tokens=64, hidden=2048, inner=1408, experts=64, first=0,
             local=64, top_k=6, gate="softmax", bias=False),
        # one decoded token through a projection with its request's adapter
        dict(name="adapters_token", op="adapters", tokens=1, d_in=7168, d_out=2048, rank=16, adapters=8,
             segment=1, none=0.0),
        # a decode batch, each request with an adapter of its own or none, at the wide projection
        dict(name="adapters_decode", op="adapters", tokens=48, d_in=7168, d_out=18432, rank=32, adapters=64,
             segment=1, none=0.1),
        # prompts of several requests in one batch, odd lengths, a higher rank
        dict(name="adapters_ragged", op="adapters", tokens=1333, d_in=2048, d_out=7168, rank=64, adapters=5,
             segment=97, none=0.2),
        # the wide projection on 4096 prompt tokens
        dict(name="adapters_prompt", op="adapters", tokens=4096, d_in=7168, d_out=18432, rank=16, adapters=8,
             segment=512, none=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_grad", "experts", "experts", "adapters", "adapters"])
    if kind in ("norm", "norm_grad"):
        cols = _log_int(rng, 64, 12288)
        quant = kind == "norm" and rng.random() < 0.4
        if quant:
            cols = 128 * max(1, cols // 128)
        elif rng.random() < 0.5:
            cols = 8 * max(1, cols // 8)
        rows = _log_int(rng, 1, max(2, min(20000, 8192 * 7168 // cols)))
        case = dict(op=kind, rows=rows, cols=cols, x=rng.choice(["bf16", "fp32"] if rows * cols <= 8192 * 3584 else ["bf16"]),
                    w=rng.choice(["bf16", "fp32"]))
        if kind == "norm":
            case["quant"] = quant
        return case
    if kind == "experts":
        hidden = 128 * _log_int(rng, 4, 56)
        inner = 128 * _log_int(rng, 1, 16)
        experts = rng.randint(2, 64)
        local = rng.randint(1, experts)
        local = max(1, min(local, 8 * 7168 * 2048 // (hidden * inner)))
        return dict(op="experts", tokens=_log_int(rng, 1, 64), hidden=hidden, inner=inner, experts=experts,
                    first=rng.randint(0, experts - local), local=local, top_k=rng.randint(1, min(8, experts)),
                    **rng.choice([dict(gate="softmax", bias=False), dict(gate="sigmoid", bias=False),
                                  dict(gate="sigmoid", bias=True)]))
    d_in = 128 * _log_int(rng, 4, 56)
    d_out = 128 * _log_int(rng, 4, 128)
    rank = 8 * rng.randint(1, 8)
    return dict(op="adapters", tokens=_log_int(rng, 1, 4096), d_in=d_in, d_out=d_out, rank=rank,
                adapters=rng.randint(1, min(64, 1024 // rank)), segment=_log_int(rng, 1, 512), none=rng.choice([0.0, 0.2]))


# ---------------------------------------------------------------- inputs

def _activations(g, rows, cols, dtype):
    """N(0, 1) with 16 outlier channels, as the quantizer's inputs have."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    ch = torch.randperm(cols, generator=g, device=DEV)[:16]
    boost = torch.where(torch.rand(rows, ch.numel(), generator=g, device=DEV) < 0.3, 20.0, 1.0)
    x[:, ch] = x[:, ch] * boost
    return x.to(dtype)


def _weight_codes(g, lead, rows, cols):
    """Gaussian BF16 weights quantized in 128x128 blocks: operand-tiled E4M3
    codes [lead][rows][cols] and FP32 block scales [lead][rows/128][cols/128]."""
    w = (torch.randn(lead, rows, cols, generator=g, device=DEV) * 0.02).bfloat16().float()
    b = w.view(lead, rows // 128, 128, cols // 128, 128)
    s = (b.abs().amax(dim=(2, 4)) / E4M3_MAX).clamp_min(SCALE_FLOOR)
    q = (b / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    # rows (r/16, r%16), columns (c/128, half of the 128, c/16 in the half, c%16)
    q = q.view(lead, rows // 16, 16, cols // 128, 2, 4, 16).permute(0, 1, 3, 4, 5, 2, 6)
    return q.reshape(lead, rows, cols), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        dt, wdt = _DT[case["x"]], _DT[case["w"]]
        rows, cols = case["rows"], case["cols"]
        s = dict(case=case, x=_activations(g, rows, cols, dt),
                 weight=(1.0 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(wdt),
                 bias=(0.1 * torch.randn(cols, generator=g, device=DEV)).to(wdt))
        if op == "norm_grad":
            s["dy"] = (1e-3 * torch.randn(rows, cols, generator=g, device=DEV)).to(dt)
            xf = s["x"].float()
            s["mean"] = xf.mean(dim=1)
            s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(dim=1) + EPS)
        return s
    if op == "experts":
        h, i, e = case["hidden"], case["inner"], case["experts"]
        w13, s13 = _weight_codes(g, case["local"], 2 * i, h)
        w2, s2 = _weight_codes(g, case["local"], h, i)
        x = _activations(g, case["tokens"], h, torch.bfloat16)
        router = (torch.randn(e, h, generator=g, device=DEV) / math.sqrt(h)).bfloat16()
        bias = 0.05 * torch.randn(e, generator=g, device=DEV) if case["bias"] else None
        return dict(case=case, x=x, router=router, w13=w13, s13=s13, w2=w2, s2=s2, bias=bias)
    t, k, n, r, a = case["tokens"], case["d_in"], case["d_out"], case["rank"], case["adapters"]
    w, sw = _weight_codes(g, 1, n, k)
    segments = (t + case["segment"] - 1) // case["segment"]
    ids = torch.randint(0, a, (segments,), generator=g, device=DEV)
    ids = torch.where(torch.rand(segments, generator=g, device=DEV) < case["none"], -1, ids)
    ids = ids.repeat_interleave(case["segment"])[:t].to(torch.int32).contiguous()
    return dict(case=case, x=_activations(g, t, k, torch.bfloat16), w=w[0], sw=sw[0],
                lora_a=(torch.randn(a, r, k, generator=g, device=DEV) / math.sqrt(k)).bfloat16(),
                lora_b=(0.1 * torch.randn(a, n, r, generator=g, device=DEV)).bfloat16(),
                ids=ids, scales=0.5 + torch.rand(a, generator=g, device=DEV))


# ---------------------------------------------------------------- plain form, FP32

def _untile(q):
    """Operand-tiled codes [..., rows, cols] -> their FP32 values, row-major."""
    lead, (rows, cols) = q.shape[:-2], q.shape[-2:]
    v = q.view(torch.float8_e4m3fn).float().view(*lead, rows // 16, cols // 128, 2, 4, 16, 16)
    n = len(lead)
    return v.permute(*range(n), n, n + 4, n + 1, n + 2, n + 3, n + 5).reshape(*lead, rows, cols)


def _dequant_weight(q, s):
    lead, (rows, cols) = q.shape[:-2], q.shape[-2:]
    v = _untile(q).view(*lead, rows // 128, 128, cols // 128, 128)
    return (v * s[..., :, None, :, None]).view(*lead, rows, cols)


def _quant_rows(x):
    """1x128 tiles of FP32 rows: E4M3 codes as FP32 values, and the scales."""
    b = x.view(*x.shape[:-1], x.shape[-1] // 128, 128)
    amax = b.abs().amax(dim=-1)
    # a tensor of 448s: dividing by a number multiplies by its rounded inverse,
    # which moves the exact ties of BF16 rows
    s = (amax / torch.full_like(amax, E4M3_MAX)).clamp_min(SCALE_FLOOR)
    q = (b / s[..., None]).to(torch.float8_e4m3fn)
    return q, s


def _through_fp8(x):
    q, s = _quant_rows(x)
    return (q.float() * s[..., None]).view(x.shape)


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    mean = x.mean(dim=1)
    d = x - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(dim=1) + EPS)
    y = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
    if not c["quant"]:
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    q, sc = _quant_rows(y)
    return {"q": q.view(c["rows"], c["cols"]), "s": sc.t().contiguous()}


def _plain_norm_grad(s):
    x, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(dim=0), "dbias": dy.sum(dim=0)}


def _plain_experts(s):
    c = s["case"]
    x = s["x"].float()
    logits = x @ s["router"].float().t()
    score = torch.softmax(logits, dim=1) if c["gate"] == "softmax" else torch.sigmoid(logits)
    value = logits if s["bias"] is None else score + s["bias"]
    ids = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    picked = torch.gather(score, 1, ids)
    gates = torch.zeros_like(score).scatter(1, ids, picked / picked.sum(dim=1, keepdim=True))
    gates = gates[:, c["first"]:c["first"] + c["local"]]
    w13 = _dequant_weight(s["w13"], s["s13"])
    au = torch.matmul(_through_fp8(x), w13.transpose(1, 2))
    del w13
    a, u = au[..., :c["inner"]], au[..., c["inner"]:]
    h = _through_fp8(a * torch.sigmoid(a) * u)
    w2 = _dequant_weight(s["w2"], s["s2"])
    y = torch.matmul(h, w2.transpose(1, 2))
    return (y * gates.t()[:, :, None]).sum(dim=0).bfloat16()


def _plain_adapters(s):
    c = s["case"]
    x = s["x"].float()
    y = _through_fp8(x) @ _dequant_weight(s["w"], s["sw"]).t()
    a, r = c["adapters"], c["rank"]
    z = (x @ s["lora_a"].float().view(a * r, -1).t()).view(-1, a, r)
    on = s["ids"][:, None] == torch.arange(a, device=z.device)
    z = torch.where(on[:, :, None], z * s["scales"][:, None], 0.0)
    y = y + z.view(-1, a * r) @ s["lora_b"].float().transpose(1, 2).reshape(a * r, -1)
    return y.bfloat16()


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "experts": _plain_experts, "adapters": _plain_adapters}


def run(s):
    c = s["case"]
    if not own:
        return _PLAIN[c["op"]](s)
    import fine_grained_fp8_amd as fp8
    if c["op"] == "norm":
        if c["quant"]:
            q, sc = fp8.layer_norm_quant(s["x"], s["weight"], s["bias"], eps=EPS)
            return {"q": q.view(torch.float8_e4m3fn), "s": sc[:, :c["rows"]]}
        y, mean, rstd = fp8.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, return_stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if c["op"] == "norm_grad":
        dx, dw, db = fp8.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if c["op"] == "experts":
        return fp8.moe_few_tokens(s["x"], s["router"], s["w13"], s["s13"], s["w2"], s["s2"], top_k=c["top_k"],
                                  gate=c["gate"], bias=s["bias"], first_expert=c["first"])
    return fp8.adapter_linear(s["x"], s["w"], s["sw"], s["lora_a"], s["lora_b"], s["ids"], scales=s["scales"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n = case["rows"] * case["cols"]
        e = 2 if case["x"] == "bf16" else 4
        we = 2 if case["w"] == "bf16" else 4
        if op == "norm_grad":
            return {"bytes": 3 * e * n + 8 * case["rows"] + (we + 8) * case["cols"], "flops": 12 * n}
        if case["quant"]:
            return {"bytes": (e + 1) * n + n // 32 + 2 * we * case["cols"], "flops": 10 * n}
        return {"bytes": 2 * e * n + 8 * case["rows"] + 2 * we * case["cols"], "flops": 8 * n}
    if op == "experts":
        t, h, i, e, k, loc = (case[v] for v in ("tokens", "hidden", "inner", "experts", "top_k", "local"))
        touched = loc * (1.0 - (1.0 - k / e) ** t)      # experts held here that some token chose, on average
        pairs = t * k * loc / e
        weights = touched * 3 * h * i * (1 + 4 / 16384)
        return {"bytes": weights + 2 * e * h + 4 * t * h, "flops": 6 * h * i * pairs + 2 * t * e * h}
    t, k, n, r, a = (case[v] for v in ("tokens", "d_in", "d_out", "rank", "adapters"))
    segments = (t + case["segment"] - 1) // case["segment"]
    touched = a * (1.0 - (1.0 - (1.0 - case["none"]) / a) ** segments)
    return {"bytes": n * k * (1 + 4 / 16384) + 2 * t * (k + n) + touched * 2 * r * (k + n) + 4 * t,
            "flops": 2 * t * n * k + 2 * t * (1.0 - case["none"]) * r * (k + n)}


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


def _weights64(q, s):
    """FP64 weights [rows][cols] of one operand-tiled matrix."""
    rows, cols = q.shape
    r = torch.arange(rows, device=q.device)[:, None]
    c = torch.arange(cols, device=q.device)[None, :]
    at = ((r // 16) * (cols // 128) + c // 128) * 2048 + ((c % 128) // 64) * 1024
    at = at + (((c % 64) // 16) * 16 + r % 16) * 16 + c % 16
    return _values_of_codes(q.reshape(-1)[at]) * s.double()[r // 128, c // 128]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    x = s["x"].double()
    if op in ("norm", "norm_grad"):
        w = s["weight"].double()
        if op == "norm":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + EPS) ** -0.5
            y = (x - mean[:, None]) * rstd[:, None] * w + s["bias"].double()
            if not case["quant"]:
                return {"y": y, "mean": mean, "rstd": rstd}
            q, sc = _tiles64(y)
            return {"q": q.reshape(y.shape), "s": sc.t().contiguous()}
        dy = s["dy"].double()
        mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
        xhat = (x - mean) * rstd
        gw = dy * w
        c1, c2 = gw.sum(1, keepdim=True) / case["cols"], (gw * xhat).sum(1, keepdim=True) / case["cols"]
        return {"dx": rstd * (gw - c1 - xhat * c2), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}
    if op == "experts":
        t, k, first, inner = case["tokens"], case["top_k"], case["first"], case["inner"]
        logits = x @ s["router"].double().t()
        score = 1.0 / (1.0 + torch.exp(-logits))
        if case["gate"] == "softmax":
            score = torch.exp(logits - logits.amax(1, keepdim=True))
            score = score / score.sum(1, keepdim=True)
        value = logits if s["bias"] is None else score + s["bias"].double()
        # rank of each expert: how many come before it
        e = torch.arange(case["experts"], device=x.device)
        before = (value[:, None, :] > value[:, :, None]) | ((value[:, None, :] == value[:, :, None]) & (e[None, None, :] < e[None, :, None]))
        chosen = before.sum(2) < k
        gates = torch.where(chosen, score, 0.0)
        gates = gates / gates.sum(1, keepdim=True)
        q, sx = _tiles64(x)
        xq = (q * sx[..., None]).reshape(t, -1)
        y = torch.zeros_like(x)
        for j in range(case["local"]):
            rows = torch.nonzero(chosen[:, first + j]).flatten()
            if rows.numel() == 0:
                continue
            au = xq[rows] @ _weights64(s["w13"][j], s["s13"][j]).t()
            a, u = au[:, :inner], au[:, inner:]
            qh, sh = _tiles64(a / (1.0 + torch.exp(-a)) * u)
            out = (qh * sh[..., None]).reshape(rows.numel(), -1) @ _weights64(s["w2"][j], s["s2"][j]).t()
            y[rows] += gates[rows, first + j][:, None] * out
        return y
    q, sx = _tiles64(x)
    y = (q * sx[..., None]).reshape(x.shape) @ _weights64(s["w"], s["sw"]).t()
    for a in range(case["adapters"]):
        rows = torch.nonzero(s["ids"] == a).flatten()
        if rows.numel():
            z = (x[rows] @ s["lora_a"][a].double().t()) * s["scales"][a].double()
            y[rows] += z @ s["lora_b"][a].double().t()
    return y
