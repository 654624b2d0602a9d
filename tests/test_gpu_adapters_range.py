"""Adapters whose values between the two products reach the end of fp32's range, which is past bf16's."""
import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.mark.parametrize("t", [F32, BF])
@pytest.mark.parametrize("m", [3, 700])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_between_the_products(m, t, sign):
    """V = 255 * 2^120 + p 2^118 for p = 0 .. 3: exact in fp32, the last two past where bf16 rounds to infinity, times 2^-100.
    D = V 2^-100 then is exact in fp32 and off by its rounding in bf16.  Of a V that is infinite itself D is too."""
    n, k, r = 70, 16, 8
    x, a, b = torch.zeros(m, k, device=DEV), torch.zeros(2, r, k, device=DEV), torch.zeros(2, n, r, device=DEV)
    p = torch.arange(m, device=DEV) % 4
    x[:, 0], x[:, 1] = 2.0 ** 64, p * 2.0 ** 60
    a[0, 0, 0], a[0, 0, 1] = sign * 255 * 2.0 ** 56, sign * 2.0 ** 58
    a[1, 0, 0] = sign * 2.0 ** 64                       # V = 2^128
    b[:, :, 0] = 2.0 ** -100
    index = torch.zeros(m, dtype=torch.int32, device=DEV)
    index[1] = 1
    base = torch.zeros(m, n, dtype=t, device=DEV)
    print(f"case adapter_gemm {m}x{n}x{k} {t} sign {sign}", flush=True)
    d = fp4.adapter_gemm(base, x.to(BF), a.to(BF), b.to(BF), index)
    torch.cuda.synchronize(DEV)
    want = sign * (255 * 2.0 ** 20 + p.double() * 2.0 ** 18)[:, None].expand(m, n)
    tol = (U if t == F32 else 2.0 ** -8) * want.abs()
    some = index == 0
    assert ((d.double() - want).abs() <= tol)[some].all(), d[some].double().sub(want[some]).abs().max().item()
    assert torch.isinf(d[1]).all() and (torch.sign(d[1].float()) == sign).all()
