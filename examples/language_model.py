"""The ends of a language model on the library's operators: a block served in int8 with adapters, and a training step.

    python examples/language_model.py [--tokens M] [--width K] [--hidden N] [--vocabulary V]

``ServedBlock`` norms its input into int8 codes, runs the int8 feed-forward products and adds each request's adapter to
what the down projection gives.  ``loss_of`` is a training step's forward pass: norm, gated product, norm, and the cross
entropy over the vocabulary without its logits.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_e2m1_amd as fp4  # noqa: E402
from examples.feed_forward import weights  # noqa: E402


class ServedBlock:
    """x + its residual -> norm -> gated feed-forward block in int8, with low-rank adapters beside the down projection.

    weight [K] and wg, wu [N, K], wd [K, N] bfloat16; adapters (A [L, R, N], B [L, K, R], scales [L])."""

    def __init__(self, weight, wg, wu, wd, adapters, act="silu"):
        self.weight, self.act, self.adapters = weight, act, adapters
        self.gate, self.up, self.down = (fp4.int8_quantize(w) for w in (wg, wu, wd))

    def __call__(self, x, residual, index):
        """(y, x + residual) for x, residual [M, K]; index [M] int32: each token's adapter, -1 for none."""
        codes, scales, total = fp4.rms_norm_quantize(x, self.weight, residual=residual)
        h = fp4.w8a8_gated_gemm(codes, scales, *self.gate, *self.up, act=self.act)
        y = fp4.w8a8_gemm(*fp4.int8_quantize(h), *self.down)
        a, b, s = self.adapters
        return fp4.adapter_gemm(y, h, a, b, index, scales=s, out=y), total


def loss_of(x, params, target, act="silu"):
    """The mean loss of tokens x [M, K] against target [M] (-100: none) under params = (norm1, wg, wu, wd, norm2, head)."""
    norm1, wg, wu, wd, norm2, head = params
    h = fp4.gated_gemm(fp4.rms_norm(x, norm1), wg, wu, act=act)
    y, _ = fp4.rms_norm(h @ wd.t(), norm2, residual=x)
    return fp4.cross_entropy_gemm(y, head, target).sum() / (target != -100).sum().clamp(min=1)


def parameters(width, hidden, vocabulary, device, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    one = torch.ones(width, device=device).bfloat16()
    head = (torch.randn(vocabulary, width, generator=g, device=device) / width ** 0.5).bfloat16()
    return [one, *weights(hidden, width, device, seed), one.clone(), head]


def train(steps, tokens, width, hidden, vocabulary, lr=0.02, device="cuda:0"):
    """Plain gradient steps on one random batch; returns the loss of every step."""
    g = torch.Generator(device=device).manual_seed(1)
    x = torch.randn(tokens, width, generator=g, device=device).bfloat16()
    target = torch.randint(0, vocabulary, (tokens,), generator=g, device=device)
    target[: tokens // 4] = -100
    params = [p.requires_grad_() for p in parameters(width, hidden, vocabulary, device, seed=2)]
    losses = []
    for _ in range(steps):
        loss = loss_of(x, params, target)
        grads = torch.autograd.grad(loss, params)
        with torch.no_grad():
            for p, d in zip(params, grads):
                p -= (lr * d.float() * (p.float().norm() / d.float().norm().clamp(min=1e-20))).to(p.dtype)
        losses.append(loss.item())
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2816)
    ap.add_argument("--vocabulary", type=int, default=32000)
    a = ap.parse_args()
    dev = "cuda:0"
    g = torch.Generator(device=dev).manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    norm1, wg, wu, wd, _, _ = parameters(a.width, a.hidden, a.vocabulary, dev)
    adapters = ((rn(8, 16, a.hidden) / a.hidden ** 0.5).bfloat16(), (rn(8, a.width, 16) / 4).bfloat16(),
                torch.ones(8, device=dev))
    x, residual = rn(a.tokens, a.width).bfloat16(), rn(a.tokens, a.width).bfloat16()
    index = torch.randint(-1, 8, (a.tokens,), generator=g, device=dev).int()
    y, total = ServedBlock(norm1, wg, wu, wd, adapters)(x, residual, index)
    plain = fp4.gated_gemm(fp4.rms_norm(total, norm1), wg, wu)
    plain = fp4.adapter_gemm((plain.float() @ wd.float().t()), plain, adapters[0], adapters[1], index, scales=adapters[2])
    print(f"int8 block with adapters against the bf16 one: relative error {((y.float() - plain).norm() / plain.norm()).item():.4f}")
    losses = train(20, a.tokens, a.width, a.hidden, a.vocabulary)
    print("training loss:", " ".join(f"{v:.4f}" for v in losses[::4] + losses[-1:]))


if __name__ == "__main__":
    main()
