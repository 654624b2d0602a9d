"""Every tile of the feed-forward products, with and without a K split, against exact sums.

Operands are small integers (times a power of two), so every sum is exact in fp32 whatever its order: int8
products and the kept G and U have to equal the formula's fp32 values, and gradients the 64-bit sums rounded to
bf16 once.  A stage, slice, row or segment that is lost, doubled or taken from elsewhere changes whole units.
"""
import math

import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4
from tests import ffn_plans as plans
from tests.test_gpu_ffn import ACTS, DEV, H32, HBF, act_error, activation, codes, gen, scales, within

pytestmark = pytest.mark.gpu


def name(case):
    return "x".join(map(str, case[0])) + "-" + "-".join(str(v) for v in case[1:]).replace("'", "").replace(" ", "")


def integers(g, rows, k, most=3):
    return torch.randint(-most, most + 1, (rows, k), generator=g, device=DEV, dtype=torch.int32)


def spoiled(bytes):
    """A workspace of NaN patterns."""
    return torch.full((bytes,), 255, dtype=torch.uint8, device=DEV)


def spoil(*shapes):
    """Leaves NaN in the freed memory that results of these shapes are likely to get."""
    held = [torch.full(s, math.nan, dtype=t, device=DEV) for s, t in shapes]
    torch.cuda.synchronize(DEV)
    del held


def scaled(a, sa, b, sb):
    """The int8 product, each step in fp32 on exact sums."""
    return (a.double() @ b.double().t()).float() * sa[:, None] * sb


@pytest.mark.parametrize("case", plans.W8A8, ids=name)
def test_w8a8_gemm(case):
    (m, n, k), tile, slices = case
    print(f"case w8a8_gemm {m}x{n}x{k} {tile} {slices}", flush=True)
    assert plans.product(m, n, k, 1, 1) == (tile, slices)
    g = gen(41)
    a, sa, b, sb = codes(g, m, k), scales(g, m, 0.03), codes(g, n, k), scales(g, n, 0.001)
    want = scaled(a, sa, b, sb)
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((m, n), math.nan, dtype=dtype, device=DEV)
        fp4.w8a8_gemm(a, sa, b, sb, out=out, workspace=spoiled(fp4.w8a8_gemm_workspace_size(m, n, k)))
        torch.cuda.synchronize(DEV)
        assert torch.equal(out, want.to(dtype))


@pytest.mark.parametrize("case", plans.W8A8_GATED, ids=name)
def test_w8a8_gated_gemm(case):
    (m, n, k), tile, slices = case
    act = ACTS[(m + n) % 3]
    print(f"case w8a8_gated_gemm {m}x{n}x{k} {tile} {slices} {act}", flush=True)
    assert plans.product(m, n, k, 1, 2) == (tile, slices)
    g = gen(42)
    w = 1 / (73 * 73 * math.sqrt(k) * 0.03)
    a, sa, bg, sg, bu, su = codes(g, m, k), scales(g, m, 0.03), codes(g, n, k), scales(g, n, w), codes(g, n, k), scales(g, n, w)
    y, u = scaled(a, sa, bg, sg).double(), scaled(a, sa, bu, su).double()
    want = activation(y, act)[0] * u
    for dtype, half in ((torch.float32, 0.0), (torch.bfloat16, HBF)):
        out = torch.full((m, n), math.nan, dtype=dtype, device=DEV)
        fp4.w8a8_gated_gemm(a, sa, bg, sg, bu, su, act=act, out=out,
                            workspace=spoiled(fp4.w8a8_gated_gemm_workspace_size(m, n, k)))
        torch.cuda.synchronize(DEV)
        # y and u are the kernel's own fp32 values: the activation and one product remain
        within(out, want, (act_error(y, act) * u.abs() + (half + 2 * H32) * want.abs()) * 1.01 + 1e-30, f"{dtype}")


@pytest.mark.parametrize("case", plans.GATED, ids=name)
def test_gated_gemm(case):
    (m, n, k), tile, slices = case
    act = ACTS[(m + n) % 3]
    print(f"case gated_gemm {m}x{n}x{k} {tile} {slices} {act}", flush=True)
    assert plans.product(m, n, k, 2, 2) == (tile, slices)
    g = gen(43)
    unit = 2.0 ** -round(math.log2(4 * math.sqrt(k)))     # sums of about unit size, exact all the same
    x = integers(g, m, k).bfloat16()
    wg, wu = ((integers(g, n, k) * unit).bfloat16() for _ in range(2))
    y, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    want = activation(y, act)[0] * u
    bound = (act_error(y, act) * u.abs() + (HBF + 2 * H32) * want.abs()) * 1.01 + 1e-30
    size = fp4.gated_gemm_workspace_size(m, n, k)
    spoil(((m, n), torch.float32), ((m, n), torch.float32))
    out = torch.full((m, n), math.nan, dtype=torch.bfloat16, device=DEV)
    _, kg, ku = fp4.gated_gemm(x, wg, wu, act=act, save=True, out=out, workspace=spoiled(size))
    alone = torch.full((m, n), math.nan, dtype=torch.bfloat16, device=DEV)
    fp4.gated_gemm(x, wg, wu, act=act, out=alone, workspace=spoiled(size))
    torch.cuda.synchronize(DEV)
    assert torch.equal(kg, y.float()) and torch.equal(ku, u.float())
    within(out, want, bound, "H")
    assert torch.equal(alone, out)


def exact_gradient_inputs(g, m, n):
    """dH, G and U whose dG and dU are integers: silu is 0 to more than fp32 precision at -256 and x at 32 and 64,
    where its derivative is 1, so dG = dH U or 0 and dU = dH G or 0."""
    kept = torch.tensor([-256.0, 32.0, 64.0], device=DEV)[torch.randint(0, 3, (m, n), generator=g, device=DEV)]
    return integers(g, m, n, 2).bfloat16(), kept, integers(g, m, n).float()


def exact_gradients(dh, x, wg, wu, kept, u):
    on = kept > 0
    dg, du = dh.double() * u.double() * on, dh.double() * kept.double() * on
    x, wg, wu = x.double(), wg.double(), wu.double()
    # at most 18543 terms of 2 * 64 * 3: below 2^24, exact in fp32
    return [v.float().bfloat16() for v in (dg @ wg + du @ wu, dg.t() @ x, du.t() @ x)]


@pytest.mark.parametrize("case", plans.GRADIENTS, ids=name)
def test_gated_gemm_backward(case):
    (m, n, k), px, pw, merged = case
    print(f"case gated_gemm_backward {m}x{n}x{k} dX {px} dW {pw} {'one launch' if merged else ''}", flush=True)
    assert plans.gradients(m, n, k) == (px, pw, merged)
    g = gen(44)
    x, wg, wu = (integers(g, rows, k).bfloat16() for rows in (m, n, n))
    dh, kept, u = exact_gradient_inputs(g, m, n)
    want = exact_gradients(dh, x, wg, wu, kept, u)
    size, least = fp4.gated_gemm_backward_workspace_size(m, n, k)
    for room in (size, least):                              # `least` leaves no room for a split
        spoil(*(((rows, k), torch.bfloat16) for rows in (m, n, n)))
        got = fp4.gated_gemm_backward(dh, x, wg, wu, kept, u, workspace=spoiled(room))
        torch.cuda.synchronize(DEV)
        for what, a, b in zip(("dX", "dWg", "dWu"), got, want):
            assert torch.equal(a, b), f"{what}, {room} bytes of workspace"


def test_gradients_of_rows_past_32_bit_offsets():
    """dG and dU of 65600 x 32800 hold more than 2^31 elements in rows of 32832, so rows from 65409 on start past
    them.  All but a few of those rows of dH and three earlier ones are zero: the gradients are sums of just these."""
    m, n, k = 65600, 32800, 16
    print(f"case gated_gemm_backward {m}x{n}x{k}, few rows", flush=True)
    g = gen(45)
    rows = torch.tensor([0, 1, 32769] + list(range(m - 100, m)), device=DEV)
    x, wg, wu = (integers(g, r, k).bfloat16() for r in (m, n, n))
    dh = torch.zeros(m, n, dtype=torch.bfloat16, device=DEV)
    dh[rows] = integers(g, len(rows), n, 2).bfloat16()
    kept = torch.full((m, n), 64.0, device=DEV)
    u = torch.randint(-3, 4, (m, n), generator=g, device=DEV, dtype=torch.int8).float()
    dx, dwg, dwu = fp4.gated_gemm_backward(dh, x, wg, wu, kept, u)
    torch.cuda.synchronize(DEV)
    wx, wdg, wdu = exact_gradients(dh[rows], x[rows], wg, wu, kept[rows], u[rows])
    assert torch.equal(dx[rows], wx) and torch.equal(dwg, wdg) and torch.equal(dwu, wdu)
    rest = torch.ones(m, dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert not dx[rest].any()
    # what a wrong offset would give: the last stage of 64 rows lost, or rows from the start in place of the last
    assert not torch.equal(exact_gradients(dh[rows[:-64]], x[rows[:-64]], wg, wu, kept[rows[:-64]], u[rows[:-64]])[1], wdg)
    assert not torch.equal(exact_gradients(dh[rows], x[:len(rows)], wg, wu, kept[rows], u[rows])[1], wdg)
