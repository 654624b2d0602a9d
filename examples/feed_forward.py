"""A transformer's feed-forward block on the library's operators: served in int8, trained in bf16.

    python examples/feed_forward.py [--tokens M] [--width K] [--hidden N] [--act silu]

``Int8FeedForward`` quantizes its weights once and runs quantize -> gated product -> quantize ->
product for every call.  ``gated_product`` is the gated half, differentiable, over any leading dimensions.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_e2m1_amd as fp4  # noqa: E402


class Int8FeedForward:
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T with int8 weights (a scale for each channel) and int8
    activations (a scale for each token, found on the way).  Wg, Wu [N, K] and Wd [K, N] are
    float32 or bfloat16 on a GPU, N and K multiples of 16."""

    def __init__(self, wg, wu, wd, act="silu"):
        self.act = act
        self.gate, self.up, self.down = (fp4.int8_quantize(w) for w in (wg, wu, wd))

    def __call__(self, x):
        rows = x.reshape(-1, x.shape[-1])
        q, s = fp4.int8_quantize(rows)
        h = fp4.w8a8_gated_gemm(q, s, *self.gate, *self.up, act=self.act)
        q, s = fp4.int8_quantize(h)
        y = fp4.w8a8_gemm(q, s, *self.down)
        return y.reshape(*x.shape[:-1], y.shape[-1])


def gated_product(x, wg, wu, act="silu"):
    """act(x Wg^T) * (x Wu^T) for bf16 x [.., K], Wg and Wu [N, K], with gradients of those that require them."""
    h = fp4.gated_gemm(x.reshape(-1, x.shape[-1]), wg, wu, act=act)
    return h.reshape(*x.shape[:-1], wg.shape[0])


def weights(n, k, device, seed=0):
    """Random Wg, Wu [n, k] and Wd [k, n] in bf16, scaled to keep unit variance."""
    g = torch.Generator(device=device).manual_seed(seed)
    return tuple((torch.randn(shape, generator=g, device=device) / shape[1] ** 0.5).bfloat16()
                 for shape in ((n, k), (n, k), (k, n)))


def train(steps, tokens, n, k, act="silu", lr=0.1, device="cuda:0"):
    """Fits a block to another block's answers on one batch; returns the loss of every step."""
    x = torch.randn(tokens, k, generator=torch.Generator(device=device).manual_seed(1), device=device).bfloat16()
    tg, tu, td = weights(n, k, device, seed=2)
    target = (gated_product(x, tg, tu, act) @ td.t()).float()
    params = [w.requires_grad_() for w in weights(n, k, device, seed=3)]
    losses = []
    for _ in range(steps):
        y = gated_product(x, params[0], params[1], act) @ params[2].t()
        loss = (y.float() - target).square().mean()
        grads = torch.autograd.grad(loss, params)
        with torch.no_grad():
            for p, d in zip(params, grads):
                # the same step length whatever the gradient's scale
                p -= (lr * d.float() * (p.float().norm() / d.float().norm().clamp(min=1e-20))).to(p.dtype)
        losses.append(loss.item())
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2816)
    ap.add_argument("--act", default="silu", choices=["silu", "gelu", "gelu_tanh"])
    a = ap.parse_args()
    wg, wu, wd = weights(a.hidden, a.width, "cuda:0")
    x = torch.randn(a.tokens, a.width, device="cuda:0").bfloat16()
    served = Int8FeedForward(wg, wu, wd, a.act)(x).float()
    plain = gated_product(x, wg, wu, a.act).float() @ wd.float().t()
    print(f"int8 block against the bf16 one: relative error {((served - plain).norm() / plain.norm()).item():.4f}")
    losses = train(20, a.tokens, a.hidden, a.width, a.act)
    print("training loss:", " ".join(f"{v:.4f}" for v in losses[::4] + losses[-1:]))


if __name__ == "__main__":
    main()
