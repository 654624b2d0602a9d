"""The activations and their derivatives far from zero, relative to the value.

Pre-activations are handed over exactly: one token with the codes 1, 0, 0 .. and a scale of one gives g = x where
x is the scale of a channel, and the backward pass takes G as it is.  Tolerances are those of test_gpu_ffn.py
without their absolute part: h(fp32) (8 |z| + 10) of the value for an activation s(z) x, 64 h(fp32) (1 + |x| z')
for its derivative, h(bf16) for each rounding; and a few units of 2^-149 where values are subnormal.
"""
import math

import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4
from tests.test_gpu_ffn import DEV, H32, HBF, activation, gen, within

pytestmark = pytest.mark.gpu

TINY = 8 * 2.0 ** -149


def values(low, high, seed=51):
    x = torch.rand(4001, generator=gen(seed), device=DEV, dtype=torch.float64) * (high - low) + low
    return x.float()


def served(x, act, tokens):
    """act(x) through w8a8_gated_gemm of `tokens` equal tokens: 1 runs the few-token kernels, 65 the tiles."""
    n = x.numel()
    a = torch.zeros(tokens, 16, dtype=torch.int8, device=DEV)
    a[:, 0] = 1
    b = torch.zeros(n, 16, dtype=torch.int8, device=DEV)
    b[:, 0] = 1
    d = fp4.w8a8_gated_gemm(a, torch.ones(tokens, device=DEV), b, x, b, torch.ones(n, device=DEV), act=act,
                            out_dtype=torch.float32)
    torch.cuda.synchronize(DEV)
    assert torch.equal(d[0].view(torch.int32), d[-1].view(torch.int32))
    return d[0]


def gradients(x, act):
    """act'(x) and act(x) as gated_gemm_backward rounds them: dX of dH = U = 1 and one channel whose weights pick
    dG in the first column and dU in the second."""
    m = x.numel()
    wg, wu = torch.zeros(1, 8, device=DEV).bfloat16(), torch.zeros(1, 8, device=DEV).bfloat16()
    wg[0, 0] = wu[0, 1] = 1
    one = torch.ones(m, 1, device=DEV)
    rows = torch.zeros(m, 8, device=DEV).bfloat16()
    dx, _, _ = fp4.gated_gemm_backward(one.bfloat16(), rows, wg, wu, x[:, None].contiguous(), one, act=act)
    torch.cuda.synchronize(DEV)
    return dx[:, 0], dx[:, 1]


# silu(x) is a normal fp32 number down to x = -91.9, where s(x) has long left their range
@pytest.mark.parametrize("act,low,high", [("silu", -91.8, -86.0), ("silu", -86.0, -20.0), ("silu", -20.0, 100.0),
                                          ("gelu_tanh", -10.1, -9.5), ("gelu_tanh", -9.5, 20.0)])
def test_sigmoid_activations(act, low, high):
    print(f"case {act} {low} .. {high}", flush=True)
    x = values(low, high)
    a, da, z, dz = activation(x.double(), act)
    for tokens in (1, 65):
        within(served(x, act, tokens), a, H32 * a.abs() * (8 * z.abs() + 10) + TINY, f"{act} of {tokens} tokens")
    got, kept = gradients(x, act)
    s = torch.sigmoid(z)
    # the derivative's two terms may cancel: relative to their magnitudes
    terms = s * (1 + (x.double() * torch.sigmoid(-z) * dz).abs())
    slope = 64 * H32 * (1 + (x.double() * dz).abs())
    within(got, da, (2 * HBF * da.abs() + slope * terms) * 1.01 + 1e-38, f"{act}'")
    within(kept, a, (2 * HBF + H32 * (8 * z.abs() + 12)) * 1.01 * a.abs() + 1e-38, f"{act} in dU")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_ends_of_the_type(act):
    """Largest values, zeros, infinities and NaN."""
    print(f"case {act}, ends of fp32", flush=True)
    most = torch.finfo(torch.float32).max
    x = torch.tensor([0.0, -0.0, most, -most, 1e30, -1e30, 200.0, -200.0, math.inf, math.nan], device=DEV)
    want = [0.0, 0.0, most, 0.0, float(x[4]), 0.0, 200.0, 0.0, math.inf]
    for tokens in (1, 65):
        got = served(x, act, tokens)
        assert got[:9].tolist() == want and torch.isnan(got[9])
    # (act(most) is infinite in bf16 and would meet a zero weight in the sum)
    slope, _ = gradients(x[[0, 1, 3, 4, 5, 6, 7, 9]], act)
    assert slope[:7].tolist() == [0.5, 0.5, 0.0, 1.0, 0.0, 1.0, 0.0] and torch.isnan(slope[7])


# gelu is a normal fp32 number down to x = -13.1
@pytest.mark.parametrize("low,high", [(-13.1, -9.0), (-9.0, -5.0), (-5.0, -1.0), (-1.0, 30.0)])
def test_erf_activation(low, high):
    """erfc amplifies the rounding of its argument and of the constant 1/sqrt 2 (1.5 h(fp32) together) by at most
    x^2 + 2, is itself off by 16 units at most (32 h(fp32)), and is subnormal below x = -12.9."""
    print(f"case gelu {low} .. {high}", flush=True)
    x = values(low, high)
    a, da, _, _ = activation(x.double(), "gelu")
    relative = H32 * (2 * x.double() ** 2 + 40)
    for tokens in (1, 65):
        within(served(x, "gelu", tokens), a, relative * a.abs() + 4 * TINY, f"gelu of {tokens} tokens")
    got, kept = gradients(x, "gelu")
    terms = da.abs() + 2 * (x.double() * torch.exp(-0.5 * x.double() ** 2)).abs() / math.sqrt(2 * math.pi)
    within(got, da, (2 * HBF * da.abs() + (relative + 24 * H32) * terms) * 1.01 + 1e-38, "gelu'")
    within(kept, a, (2 * HBF + relative) * 1.01 * a.abs() + 1e-38, "gelu in dU")
