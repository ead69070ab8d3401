"""One decoder block around the FP8 products, served and trained with the
library's operators.

    python examples/decoder_block.py [--hidden 7168] [--inner 2048] [--tokens 32]

serve(): a batch of requests, each with a low-rank adapter of its own or none,
through layer norm, the shared FP8 projection with the adapters, layer norm,
and the mixture-of-experts layer.  The same call takes one decoded token per
request or their prompts; the expert layer takes up to 64 tokens at a time.

train_step(): layer norm with the fused 1x128 quantization into the FP8 Fprop
product, and back: Dgrad and Wgrad on FP8 codes, then the norm's gradients.

Random weights; needs an MI355X and the built library.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fine_grained_fp8_amd as fp8  # noqa: E402


def quantized(rows, cols, count=None, std=0.02):
    """Random BF16 weights as operand-tiled codes and block scales ([count] of them)."""
    made = [fp8.quant_weight_128x128((std * torch.randn(rows, cols, device="cuda")).bfloat16(), tiled=True)[:2]
            for _ in range(count or 1)]
    if count is None:
        return made[0]
    return torch.stack([q for q, _ in made]), torch.stack([s for _, s in made])


class Block:
    def __init__(self, hidden, inner, experts=8, adapters=4, rank=16, top_k=2):
        self.hidden, self.top_k = hidden, top_k
        self.norm1 = torch.ones(hidden, device="cuda"), torch.zeros(hidden, device="cuda")
        self.norm2 = torch.ones(hidden, device="cuda"), torch.zeros(hidden, device="cuda")
        self.w, self.sw = quantized(hidden, hidden)
        self.lora_a = (torch.randn(adapters, rank, hidden, device="cuda") * hidden ** -0.5).bfloat16()
        self.lora_b = (torch.randn(adapters, hidden, rank, device="cuda") * 0.1).bfloat16()
        self.router = (torch.randn(experts, hidden, device="cuda") * hidden ** -0.5).bfloat16()
        self.w13, self.s13 = quantized(2 * inner, hidden, experts)
        self.w2, self.s2 = quantized(hidden, inner, experts)

    def experts(self, x):
        """The expert layer, 64 tokens at a time."""
        parts = [fp8.moe_few_tokens(p, self.router, self.w13, self.s13, self.w2, self.s2, top_k=self.top_k)
                 for p in x.split(64)]
        return parts[0] if len(parts) == 1 else torch.cat(parts)

    def serve(self, x, ids):
        """x bfloat16 [tokens][hidden], ids int32 [tokens]: each token's adapter (-1: none)."""
        x = x + fp8.adapter_linear(fp8.layer_norm(x, *self.norm1), self.w, self.sw, self.lora_a, self.lora_b, ids)
        return x + self.experts(fp8.layer_norm(x, *self.norm2))


def train_step(x, norm, w_bf16, dy):
    """y = W norm(x) and its gradients (dx, dW, dnorm_weight, dnorm_bias) on FP8
    products; rows a multiple of 128."""
    w, sw, wt = fp8.quant_weight_128x128(w_bf16, transposed=True, tiled=True)
    q, s, n, mean, rstd = fp8.layer_norm_quant(x, *norm, return_y=True, return_stats=True)
    y = fp8.block_gemm("fprop_tiled", q, s, w, sw)
    dq, ds, dqt, dst = fp8.quant_act_dual(dy)
    nt, nst, _ = fp8.quant_act_1x128(n, "col_tiled")
    dw = fp8.block_gemm("wgrad_tiled", dqt, dst, nt, nst, out_dtype=torch.float32)
    dn = fp8.block_gemm("dgrad_t_tiled", dq, ds, wt, sw)
    dx, dnorm_w, dnorm_b = fp8.layer_norm_backward(dn, x, mean, rstd, norm[0])
    return y, dx, dw, dnorm_w, dnorm_b


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--tokens", type=int, default=32)
    args = ap.parse_args()
    torch.manual_seed(0)
    block = Block(args.hidden, args.inner)
    x = torch.randn(args.tokens, args.hidden, device="cuda").bfloat16()
    ids = (torch.arange(args.tokens, device="cuda") % 5 - 1).to(torch.int32)
    block.serve(x, ids)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        y = block.serve(x, ids)
    end.record()
    torch.cuda.synchronize()
    print(f"serve {args.tokens} tokens: {start.elapsed_time(end) / 10 * 1e3:.1f} us a block, |y| {y.float().abs().mean():.3f}")
    rows = 1024
    x = torch.randn(rows, args.hidden, device="cuda").bfloat16()
    w = (0.02 * torch.randn(args.hidden, args.hidden, device="cuda")).bfloat16()
    dy = (1e-3 * torch.randn(rows, args.hidden, device="cuda")).bfloat16()
    out = train_step(x, block.norm1, w, dy)
    torch.cuda.synchronize()
    print("train step: " + ", ".join(f"{n} {tuple(t.shape)}" for n, t in zip(("y", "dx", "dw", "dnorm_w", "dnorm_b"), out)))


if __name__ == "__main__":
    main()
