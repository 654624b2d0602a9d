"""The loss and its gradients where logits are large beside their differences.

Logits here are exact in fp32 (one or two products of few bits), so what is left is the rounding of the softmax itself, which
turns on differences of logits alone, not on their size.  u = 2^-24 is the half step of fp32.
"""
import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4
from tests import loss_plans as plans

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
TOPS = (20, 300, 3000)
# One size for each of the forward product's tiles, as every row is taken and as rows are gathered.
SIZES = [(67, 2023, 456), (71, 68, 8240), (664, 4894, 72), (386, 26319, 72), (5000, 66, 72), (4200, 30000, 72)]


def confident(m, v, k, top):
    """Row i knows its token: its logit is about `top`, every other minus that."""
    g = torch.Generator(device=DEV).manual_seed(top)
    x, w = torch.zeros(m, k, device=DEV), torch.zeros(v, k, device=DEV)
    x[:, 3] = (top * (1 + 0.5 * torch.rand(m, generator=g, device=DEV))).bfloat16().float()
    w[:, 3] = -1
    at = v - 2
    w[at, 3] = 1
    t = torch.full((m,), at, device=DEV)
    t[::7] = -100
    return x.bfloat16(), w.bfloat16(), t


def test_the_sizes_are_those_of_every_tile():
    assert {plans.products(*s)[0] for s in SIZES} == {"256", "128", "64x128", "64x128Long"}


@pytest.mark.parametrize("top", TOPS)
@pytest.mark.parametrize("m,v,k", SIZES)
def test_a_confident_token_has_no_loss(m, v, k, top):
    """Every other token's share is below V e^-40, less than half a step of 1, so that the sum of exponentials is 1, its
    logarithm 0, the loss 0 and lse the logit itself; one step of the sum, 2^-23, is allowed upwards and nothing downwards."""
    print(f"case cross_entropy_gemm {m}x{v}x{k} logits of {top}", flush=True)
    x, w, t = confident(m, v, k, top)
    loss, lse = fp4.cross_entropy_gemm(x, w, t, save=True)
    torch.cuda.synchronize(DEV)
    z = torch.where(t == -100, torch.zeros_like(lse), x[:, 3].float())
    assert (loss >= 0).all(), f"a loss of {loss.min().item():.3g}"
    assert (loss <= 2 * U).all(), f"a loss of {loss.max().item():.3g}"
    assert ((lse - z).abs() <= 2 * U * (1 + z)).all()


@pytest.mark.parametrize("top", [16, 256, 4096])
@pytest.mark.parametrize("m,v,k", SIZES)
def test_the_loss_goes_by_differences(m, v, k, top):
    """Logits top + d with d = 0, -1/16, .. -16: exact, and so are their differences.  A term e^d takes an exponent of two
    roundings, its own rounding and, where parts are joined, the same again: (4 |d| + 8) u of it; the sum's chains have at most
    V / 1024 + 80 additions; the logarithm and the last additions round numbers of the loss's size and of the span."""
    print(f"case cross_entropy_gemm {m}x{v}x{k} logits from {top}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(top + 1)
    x, w = torch.zeros(m, k, device=DEV), torch.zeros(v, k, device=DEV)
    x[:, 0], x[:, 5] = top, 1
    w[:, 0] = 1
    w[:, 5] = -torch.randint(0, 256, (v,), generator=g, device=DEV).float() / 16
    t = torch.randint(0, v, (m,), generator=g, device=DEV)
    loss = fp4.cross_entropy_gemm(x.bfloat16(), w.bfloat16(), t)
    torch.cuda.synchronize(DEV)
    d = w[:, 5].double()
    want = torch.logsumexp(d, 0) - d[t]
    tol = (v / 1024 + 100 + 4 * 16) * U + 8 * U * (want + 16)
    err = (loss.double() - want).abs()
    assert (err <= tol).all(), f"off by {err.max().item():.3g}, allowed {tol.max().item():.3g}"


@pytest.mark.parametrize("top", TOPS)
@pytest.mark.parametrize("m,v,k", [s for s in SIZES if s[1] != 66] + [(200, 66, 528), (129, 2000, 136)])
def test_a_confident_token_has_no_gradient(m, v, k, top):
    """lse is the wanted logit itself and so exact: p - 1 is 0, but for one step of the exponential, and the other
    tokens' p are below e^-40.  P is then at most 2 u dL + V e^-40 dL and what it gives, with weights of 1 and rows of
    1.5 top, at most that many times over."""
    print(f"case cross_entropy_gemm_backward {m}x{v}x{k} logits of {top}", flush=True)
    x, w, t = confident(m, v, k, top)
    lse = torch.where(t == -100, torch.full_like(x[:, 3], 7), x[:, 3]).float()
    dx, dw = fp4.cross_entropy_gemm_backward(torch.ones(m, device=DEV), x, w, t, lse)
    torch.cuda.synchronize(DEV)
    assert dx.float().abs().max() <= 2.5 * U, dx.float().abs().max().item()
    assert dw.float().abs().max() <= 2.5 * U * 1.5 * top * m, dw.float().abs().max().item()
