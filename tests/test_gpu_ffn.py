"""The feed-forward operators on the GPU against their formulas in 64 bits.

Tolerances.  Let h(t) be half a step of type t relative to the value (bf16 2^-8, fp32 2^-24).
  * int8 sums are exact, so a scaled product is off by the rounding of the sum to fp32 and
    two fp32 products: 3 h(fp32) |D|, and h(out) more for a bf16 result.
  * bf16 products are exact in fp32 and a sum of K of them in any order is off by at most
    K 2 h(fp32) sum|x||w| (the factor 2 covers a matrix unit that truncates).
  * an activation adds E_a = h(fp32) |a| (8 |z| + 10) from 2^x, the reciprocal and z (z = x
    for silu, the cubic for gelu_tanh), or 8 h(fp32) |x| for erf; its derivative adds
    64 h(fp32) (1 + |x| z').
  * gradients: dG and dU are rounded to bf16 once, then summed like any bf16 product, and
    rounded once more.
"""
import math

import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
H32, HBF = 2.0 ** -24, 2.0 ** -8
ACTS = ["silu", "gelu", "gelu_tanh"]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def codes(g, rows, k):
    return torch.randint(-127, 128, (rows, k), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)


def scales(g, n, typical):
    return torch.exp(0.3 * torch.randn(n, generator=g, device=DEV)) * typical


def activation(x, act):
    """a(x), a'(x), z and z' in x's type."""
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-x * math.sqrt(0.5))
        return x * cdf, cdf + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi), x, torch.ones_like(x)
    c = 2 * math.sqrt(2 / math.pi)
    z = x if act == "silu" else c * (x + 0.044715 * x ** 3)
    dz = torch.ones_like(x) if act == "silu" else c * (1 + 3 * 0.044715 * x * x)
    s = torch.sigmoid(z)
    return x * s, s + x * s * torch.sigmoid(-z) * dz, z, dz


def act_error(x, act):
    a, _, z, _ = activation(x, act)
    return 8 * H32 * x.abs() if act == "gelu" else H32 * a.abs() * (8 * z.abs() + 10) + 1e-30


def gated_bound(g, eg, u, eu, act, half_out):
    """Bound of act(g) u for sums off by eg and eu."""
    a, da, _, _ = activation(g, act)
    ea = 1.2 * eg * 1.2 + act_error(g, act)             # |a'| <= 1.13 everywhere
    return u.abs() * ea + a.abs() * eu + ea * eu + (half_out + 2 * H32) * (a * u).abs() * 1.01


def within(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = ((got - want).abs() / bound.clamp(min=1e-300)).max().item() if got.numel() else 0.0
    print(f"{what}: worst error / bound = {over:.3g}", flush=True)
    assert over <= 1.0, f"{what}: {over}"


# ---- int8_quantize -------------------------------------------------------------------------

def quantize_reference(x):
    """The rule, with IEEE fp32 steps formed in 64 bits and rounded to 32."""
    x = x.double()
    scale = (x.abs().amax(dim=1) / 127).float()
    inv = (1 / scale.double()).float().clamp(max=torch.finfo(torch.float32).max).double()
    return (x * inv[:, None]).float().double().round().clamp(-127, 127).to(torch.int8), scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,k", [(1, 16), (3, 256), (5, 272), (7, 528), (130, 1040), (9, 2064), (4, 4096), (33, 8208),
                                    (3, 16400), (2, 32784), (3, 65552), (1, 131088)])
def test_quantize(rows, k, dtype):
    print(f"case int8_quantize {rows}x{k} {dtype}", flush=True)
    x = (torch.randn(rows, k, generator=gen(rows + k), device=DEV) *
         torch.exp(torch.randn(rows, 1, generator=gen(k), device=DEV))).to(dtype)
    c, s = fp4.int8_quantize(x)
    torch.cuda.synchronize(DEV)
    rc, rs = quantize_reference(x)
    assert torch.equal(s, rs)
    assert torch.equal(c, rc)


@pytest.mark.parametrize("k", [64, 1024, 16384, 131072])
def test_quantize_special_rows(k):
    """Zeros, ties, subnormals, the type's extremes; infinities and NaN spoil their own row only."""
    print(f"case int8_quantize special rows k={k}", flush=True)
    x = torch.randn(12, k, generator=gen(k), device=DEV)
    x[0] = 0
    x[1] = -0.0
    x[2, :16] = torch.arange(16, device=DEV) + 0.5      # with 127 as the maximum: ties at scale 1
    x[2, 16] = 127.0
    x[2, 17:] = 0
    x[3] = 1e-45                                        # smallest subnormal: 1/scale overflows
    x[4] *= 1e-41
    x[5, k - 1] = -torch.finfo(torch.float32).max
    x[6, k // 2] = math.inf
    x[7, 0] = -math.inf
    x[8, k - 1] = math.nan
    c, s = fp4.int8_quantize(x)
    torch.cuda.synchronize(DEV)
    fine = [0, 1, 2, 3, 4, 5, 9, 10, 11]
    rc, rs = quantize_reference(x[fine])
    rc[rs == 0] = 0
    assert torch.equal(s[fine], rs)
    assert torch.equal(c[fine], rc)
    assert torch.isnan(s[[6, 7, 8]]).all() and not c[[6, 7, 8]].any()


def test_quantize_empty():
    c, s = fp4.int8_quantize(torch.empty((0, 64), device=DEV))
    assert c.shape == (0, 64) and s.shape == (0,)
    c, s = fp4.int8_quantize(torch.empty((5, 0), device=DEV))
    torch.cuda.synchronize(DEV)
    assert c.shape == (5, 0) and not s.any()


# ---- products of int8 operands -------------------------------------------------------------

# One token to many, odd sizes, K below, at and past a stage, every tile and the K split.
INT8 = [(1, 1, 16), (1, 4096, 4096), (2, 33, 16), (7, 130, 144), (8, 1000, 2064), (16, 515, 8192), (17, 64, 4112),
        (33, 257, 1040), (64, 700, 16384), (100, 129, 10000), (129, 2048, 128), (257, 1117, 272), (300, 4096, 4096),
        (1003, 1117, 1040), (2100, 4099, 528)]


def int8_inputs(m, n, k, seed, weights):
    g = gen(seed)
    return (codes(g, m, k), scales(g, m, 0.03)) + tuple(
        t for _ in range(weights) for t in (codes(g, n, k), scales(g, n, 1 / (73 * 73 * math.sqrt(k) * 0.03))))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", INT8)
def test_w8a8_gemm(m, n, k, out):
    print(f"case w8a8_gemm {m}x{n}x{k} {out}", flush=True)
    a, sa, b, sb = int8_inputs(m, n, k, 1, 1)
    want = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
    bound = want.abs() * (3 * H32 + (HBF if out is torch.bfloat16 else 0)) * 1.01
    for space in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):     # with and without a split
        d = fp4.w8a8_gemm(a, sa, b, sb, out_dtype=out, workspace=space)
        torch.cuda.synchronize(DEV)
        assert d.dtype is out
        within(d, want, bound + 1e-40, f"w8a8_gemm {m}x{n}x{k}")


# Every token packing (up to 4, 8, 16, 32, 64) at weights that stream past the caches (32 MB
# and more) and at few rows with K long enough for a split; the last group of rows is ragged.
FEW = [(m, n, k) for m in (1, 3, 4, 5, 8, 9, 16, 18, 32, 33, 47, 64) for n, k in ((8201, 4112), (70, 16400))]


@pytest.mark.parametrize("m,n,k", FEW)
def test_few_tokens(m, n, k):
    print(f"case few tokens {m}x{n}x{k}", flush=True)
    a, sa, bg, sg, bu, su = int8_inputs(m, n, k, 21, 2)
    g = (a.double() @ bg.double().t()) * sa.double()[:, None] * sg.double()
    u = (a.double() @ bu.double().t()) * sa.double()[:, None] * su.double()
    want = activation(g, "silu")[0] * u
    bound = gated_bound(g, 3 * H32 * g.abs(), u, 3 * H32 * u.abs(), "silu", 0) + 1e-30
    for space in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        one = fp4.w8a8_gemm(a, sa, bg, sg, out_dtype=torch.float32, workspace=space)
        both = fp4.w8a8_gated_gemm(a, sa, bg, sg, bu, su, out_dtype=torch.float32, workspace=space)
        torch.cuda.synchronize(DEV)
        within(one, g, 3 * H32 * g.abs() * 1.01 + 1e-40, "w8a8_gemm")
        within(both, want, bound, "w8a8_gated_gemm")


@pytest.mark.parametrize("m", [1, 3, 4, 7, 8, 15, 30, 64])
def test_few_tokens_keep_non_finite_values_apart(m):
    """Packed tokens share an instruction: a spoiled one must reach neither its neighbours nor,
    through rows past N and tokens past M, anything else."""
    for n, k in ((70, 1032), (2051, 4104)):
        print(f"case few tokens, non-finite {m}x{n}x{k}", flush=True)
        x, wg, wu, _ = bf16_inputs(m, n, k, 22)
        clean = fp4.gated_gemm(x, wg, wu)
        bad = m // 2
        x[bad, k - 1] = math.nan
        wu[n - 1, 3] = math.inf
        h, g, u = fp4.gated_gemm(x, wg, wu, save=True)
        torch.cuda.synchronize(DEV)
        rows = [i for i in range(m) if i != bad]
        assert torch.isnan(h[bad]).all() and torch.isnan(g[bad]).all() and torch.isnan(u[bad]).all()
        assert torch.equal(h[rows][:, :n - 1], clean[rows][:, :n - 1])
        assert not torch.isfinite(u[rows][:, n - 1]).any()


def test_w8a8_gemm_largest_sums():
    """Sums at the ends of 32 bits: K = 131056 of -128 * -128 and -128 * 127."""
    k = (1 << 17) - 16
    print(f"case w8a8_gemm 3x40x{k}", flush=True)
    a = torch.full((3, k), -128, dtype=torch.int8, device=DEV)
    b = torch.full((40, k), -128, dtype=torch.int8, device=DEV)
    b[1::2] = 127
    one = torch.ones(40, device=DEV)
    d = fp4.w8a8_gemm(a, one[:3].clone(), b, one, out_dtype=torch.float32)
    torch.cuda.synchronize(DEV)
    want = (a.double() @ b.double().t())
    within(d, want, want.abs() * 3 * H32, "largest sums")


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 2048, 4096), (5, 77, 272), (16, 1000, 1024), (31, 130, 8208),
                                   (65, 515, 400), (300, 1117, 1040), (1100, 2050, 144), (2048, 4096, 256)])
def test_w8a8_gated_gemm(m, n, k, act, out):
    print(f"case w8a8_gated_gemm {m}x{n}x{k} {act} {out}", flush=True)
    a, sa, bg, sg, bu, su = int8_inputs(m, n, k, 2, 2)
    g = (a.double() @ bg.double().t()) * sa.double()[:, None] * sg.double()
    u = (a.double() @ bu.double().t()) * sa.double()[:, None] * su.double()
    want = activation(g, act)[0] * u
    bound = gated_bound(g, 3 * H32 * g.abs(), u, 3 * H32 * u.abs(), act, HBF if out is torch.bfloat16 else 0)
    for space in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        d = fp4.w8a8_gated_gemm(a, sa, bg, sg, bu, su, act=act, out_dtype=out, workspace=space)
        torch.cuda.synchronize(DEV)
        within(d, want, bound + 1e-30, f"w8a8_gated_gemm {m}x{n}x{k} {act}")


def test_scale_of_a_spoiled_token_spoils_its_row_only():
    m, n, k = 20, 300, 512
    a, sa, b, sb = int8_inputs(m, n, k, 3, 1)
    clean = fp4.w8a8_gemm(a, sa, b, sb)
    sa[7] = math.nan
    d = fp4.w8a8_gemm(a, sa, b, sb)
    torch.cuda.synchronize(DEV)
    assert torch.isnan(d[7]).all()
    keep = [i for i in range(m) if i != 7]
    assert torch.equal(d[keep], clean[keep])


# ---- the gated product in bf16 -------------------------------------------------------------

BF = [(1, 1, 8), (1, 1024, 4096), (3, 65, 72), (16, 500, 1032), (17, 64, 2056), (40, 333, 8192), (130, 130, 136),
      (301, 1003, 520), (700, 2051, 264), (2048, 4096, 128)]


def bf16_inputs(m, n, k, seed):
    g = gen(seed)
    x = torch.randn(m, k, generator=g, device=DEV).bfloat16()
    wg = (torch.randn(n, k, generator=g, device=DEV) * (1.5 / math.sqrt(k))).bfloat16()
    wu = (torch.randn(n, k, generator=g, device=DEV) / math.sqrt(k)).bfloat16()
    return x, wg, wu, torch.randn(m, n, generator=g, device=DEV).bfloat16()


def sums(x, w):
    k = x.shape[1]
    return x.double() @ w.double().t(), 2 * k * H32 * (x.double().abs() @ w.double().abs().t())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", BF)
def test_gated_gemm(m, n, k, act):
    print(f"case gated_gemm {m}x{n}x{k} {act}", flush=True)
    x, wg, wu, _ = bf16_inputs(m, n, k, 4)
    (g, eg), (u, eu) = sums(x, wg), sums(x, wu)
    want = activation(g, act)[0] * u
    bound = gated_bound(g, eg, u, eu, act, HBF) + 1e-30
    for space in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        h, kg, ku = fp4.gated_gemm(x, wg, wu, act=act, save=True, workspace=space)
        alone = fp4.gated_gemm(x, wg, wu, act=act, workspace=space)
        torch.cuda.synchronize(DEV)
        within(h, want, bound, f"gated_gemm {m}x{n}x{k} {act}")
        within(kg, g, eg + 1e-30, "G")
        within(ku, u, eu + 1e-30, "U")
        within(alone, want, bound, f"gated_gemm {m}x{n}x{k} {act}, nothing kept")


def test_non_finite_values_stay_in_their_rows_and_columns():
    """K = 72 ends inside a 64-element stage: what follows a row's end must not reach it."""
    for m, n in ((10, 70), (600, 900)):
        x, wg, wu, _ = bf16_inputs(m, n, 72, 5)
        clean = fp4.gated_gemm(x, wg, wu)
        x[4, 0] = math.nan
        x[6, 71] = math.inf
        wg[9, 0] = math.nan
        h = fp4.gated_gemm(x, wg, wu)
        torch.cuda.synchronize(DEV)
        rows = [i for i in range(m) if i not in (4, 6)]
        cols = [i for i in range(n) if i != 9]
        assert torch.isnan(h[4]).all() and torch.isnan(h[:, 9]).all()
        assert torch.equal(h[rows][:, cols], clean[rows][:, cols])


# ---- gradients -----------------------------------------------------------------------------

def gradient_reference(dh, x, wg, wu, g, u, act):
    """dX, dWg, dWu in 64 bits and the bound of each."""
    dh, x, wg, wu, g, u = (t.double() for t in (dh, x, wg, wu, g, u))
    a, da, z, dz = activation(g, act)
    dg, du = dh * u * da, dh * a
    edg = HBF * dg.abs() * 1.01 + (dh * u).abs() * 64 * H32 * (1 + g.abs() * dz)
    edu = HBF * du.abs() * 1.01 + dh.abs() * (act_error(g, act) + 2 * H32 * a.abs())
    m, n = dh.shape

    def product(p, ep, q, terms):
        v, mag = p @ q, p.abs() @ q.abs()
        return v, ep @ q.abs() + 2 * terms * H32 * mag * 1.01

    (xg, exg), (xu, exu) = product(dg, edg, wg, 2 * n), product(du, edu, wu, 2 * n)
    (vg, evg), (vu, evu) = product(dg.t(), edg.t(), x, m), product(du.t(), edu.t(), x, m)
    out = []
    for v, e in ((xg + xu, exg + exu), (vg, evg), (vu, evu)):
        out.append((v, (e + HBF * (v.abs() + e)) * 1.01 + 1e-30))
    return out


GRAD = [(1, 1, 8), (1, 300, 64), (3, 65, 72), (17, 130, 1032), (64, 64, 64), (130, 257, 136), (301, 1003, 520),
        (1100, 700, 264), (2049, 520, 1304)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", GRAD)
def test_gated_gemm_backward(m, n, k, act):
    print(f"case gated_gemm_backward {m}x{n}x{k} {act}", flush=True)
    x, wg, wu, dh = bf16_inputs(m, n, k, 6)
    _, g, u = fp4.gated_gemm(x, wg, wu, act=act, save=True)
    torch.cuda.synchronize(DEV)
    want = gradient_reference(dh, x, wg, wu, g, u, act)
    least = fp4.gated_gemm_backward_workspace_size(m, n, k)[1]
    for space in (None, torch.empty(least, dtype=torch.uint8, device=DEV)):
        got = fp4.gated_gemm_backward(dh, x, wg, wu, g, u, act=act, workspace=space)
        torch.cuda.synchronize(DEV)
        for name, d, (v, e) in zip(("dX", "dWg", "dWu"), got, want):
            within(d, v, e, f"{name} {m}x{n}x{k} {act}")


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """Sum of dH * H along a direction, by central differences of the 64-bit formula."""
    m, n, k = 50, 70, 64
    x, wg, wu, dh = bf16_inputs(m, n, k, 7)
    _, g, u = fp4.gated_gemm(x, wg, wu, act=act, save=True)
    got = fp4.gated_gemm_backward(dh, x, wg, wu, g, u, act=act)
    torch.cuda.synchronize(DEV)
    bounds = gradient_reference(dh, x, wg, wu, g, u, act)
    at = [t.double() for t in (x, wg, wu)]

    def loss(p):
        return (dh.double() * activation(p[0] @ p[1].t(), act)[0] * (p[0] @ p[2].t())).sum().item()

    rng = gen(8)
    for i in range(3):
        d = torch.randn(at[i].shape, generator=rng, device=DEV, dtype=torch.float64)
        eps = 1e-4
        up, down = (loss(at[:i] + [at[i] + e * d] + at[i + 1:]) for e in (eps, -eps))
        slope = (up - down) / (2 * eps)
        # the kept G and U are fp32: their error moves the gradient far less than dG's rounding
        assert abs((got[i].double() * d).sum().item() - slope) <= (bounds[i][1] * d.abs()).sum().item() + 1e-6 * abs(slope) + 1e-4


def test_offsets_past_32_bits():
    """More than 2^31 elements in codes, results, kept sums and gradients: first, middle and last rows."""
    m, n, k = 65600, 32800, 16
    rows, cols = [0, 32769, m - 1], [0, 16400, n - 1]
    print(f"case offsets past 32 bits: quantize {m}x{n}", flush=True)
    x = torch.randn(m, n, generator=gen(31), device=DEV, dtype=torch.bfloat16)
    c, s = fp4.int8_quantize(x)
    torch.cuda.synchronize(DEV)
    rc, rs = quantize_reference(x[rows])
    assert torch.equal(s[rows], rs) and torch.equal(c[rows], rc)
    del x, c, s
    print(f"case offsets past 32 bits: w8a8_gemm {m}x{n}x{k}", flush=True)
    a, sa, b, sb = int8_inputs(m, n, k, 32, 1)
    d = fp4.w8a8_gemm(a, sa, b, sb)
    torch.cuda.synchronize(DEV)
    want = (a[rows].double() @ b.double().t()) * sa[rows].double()[:, None] * sb.double()
    within(d[rows], want, want.abs() * (3 * H32 + HBF) * 1.01 + 1e-40, "w8a8_gemm")
    del d
    print(f"case offsets past 32 bits: gated_gemm and its gradients {m}x{n}x{k}", flush=True)
    x, wg, wu, dh = bf16_inputs(m, n, k, 33)
    h, g, u = fp4.gated_gemm(x, wg, wu, save=True)
    torch.cuda.synchronize(DEV)
    (wantg, eg), (wantu, eu) = sums(x[rows], wg), sums(x[rows], wu)
    within(g[rows], wantg, eg + 1e-30, "G")
    within(u[rows], wantu, eu + 1e-30, "U")
    within(h[rows], activation(wantg, "silu")[0] * wantu, gated_bound(wantg, eg, wantu, eu, "silu", HBF) + 1e-30, "H")
    dx, dwg, dwu = fp4.gated_gemm_backward(dh, x, wg, wu, g, u)
    torch.cuda.synchronize(DEV)
    want = gradient_reference(dh[rows], x[rows], wg, wu, g[rows], u[rows], "silu")
    within(dx[rows], *want[0], "dX")
    want = gradient_reference(dh[:, cols], x, wg[cols], wu[cols], g[:, cols], u[:, cols], "silu")
    within(dwg[cols], *want[1], "dWg")
    within(dwu[cols], *want[2], "dWu")


def test_more_rows_than_a_launch_holds():
    """2^26 and more rows of 16 for the quantizer, 2^27 and more channels for one token."""
    rows = (1 << 26) + 5
    print(f"case int8_quantize {rows}x16", flush=True)
    x = torch.randn(rows, 16, generator=gen(34), device=DEV, dtype=torch.bfloat16)
    c, s = fp4.int8_quantize(x)
    torch.cuda.synchronize(DEV)
    at = [0, (1 << 25) - 1, 1 << 25, (1 << 26) - 1, 1 << 26, rows - 1]
    rc, rs = quantize_reference(x[at])
    assert torch.equal(s[at], rs) and torch.equal(c[at], rc)
    del x, c, s
    n = (1 << 27) + 3
    print(f"case w8a8_gemm 1x{n}x16", flush=True)
    a, sa = codes(gen(35), 1, 16), scales(gen(36), 1, 0.03)
    b = torch.randint(-127, 128, (n, 16), generator=gen(37), device=DEV, dtype=torch.int8)
    sb = torch.rand(n, generator=gen(38), device=DEV) + 0.5
    d = fp4.w8a8_gemm(a, sa, b, sb, out_dtype=torch.float32)
    torch.cuda.synchronize(DEV)
    at = [0, 1, 1 << 26, (1 << 27) - 1, n - 1]
    want = (a.double() @ b[at].double().t()) * sa.double()[:, None] * sb[at].double()
    within(d[:, at], want, want.abs() * 3 * H32 * 1.01 + 1e-40, "w8a8_gemm")


def test_empty_products():
    z = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    h, g, u = fp4.gated_gemm(z(3, 0), z(5, 0), z(5, 0), save=True)
    torch.cuda.synchronize(DEV)
    assert not h.any() and not g.any() and not u.any() and h.shape == (3, 5)
    assert fp4.gated_gemm(z(0, 64), z(5, 64), z(5, 64)).shape == (0, 5)
    f = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    dx, dwg, dwu = fp4.gated_gemm_backward(z(0, 5), z(0, 64), z(5, 64), z(5, 64), f(0, 5), f(0, 5))
    torch.cuda.synchronize(DEV)
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any() and dwg.shape == (5, 64)
    dx, dwg, dwu = fp4.gated_gemm_backward(z(4, 0), z(4, 64), z(0, 64), z(0, 64), f(4, 0), f(4, 0))
    torch.cuda.synchronize(DEV)
    assert not dx.any() and dx.shape == (4, 64) and dwg.shape == (0, 64)
    i8 = lambda *s: torch.empty(s, dtype=torch.int8, device=DEV)  # noqa: E731
    d = fp4.w8a8_gemm(i8(3, 0), f(3), i8(5, 0), f(5))
    torch.cuda.synchronize(DEV)
    assert not d.any() and d.shape == (3, 5)


# ---- refusals, streams, repeats, graphs ----------------------------------------------------

def test_refusals_of_tensors():
    x, wg, wu, dh = bf16_inputs(4, 6, 64, 9)
    bad = [lambda: fp4.gated_gemm(x.half(), wg, wu), lambda: fp4.gated_gemm(x, wg[:, :32].contiguous(), wu),
           lambda: fp4.gated_gemm(x, wg, wu.cpu()), lambda: fp4.gated_gemm(x.t(), wg, wu),
           lambda: fp4.gated_gemm(x[0], wg, wu), lambda: fp4.gated_gemm(x, wg, wu, act="relu"),
           lambda: fp4.gated_gemm(x[:, :60].contiguous(), wg[:, :60].contiguous(), wu[:, :60].contiguous()),
           lambda: fp4.int8_quantize(x.half()), lambda: fp4.int8_quantize(x[:, :24].contiguous()),
           lambda: fp4.gated_gemm_backward(dh, x, wg, wu, dh, dh),
           lambda: fp4.w8a8_gemm(x, x, x, x)]
    for call in bad:
        with pytest.raises((TypeError, ValueError)):
            call()
    # an operand that starts inside a 16-byte line
    flat = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(fp4.Fp4GemmError):
        fp4.gated_gemm(flat[4:4 + 256].view(4, 64), wg, wu)
    with pytest.raises(fp4.Fp4GemmError):
        fp4.gated_gemm_backward(dh, x, wg, wu, torch.zeros(4, 6, device=DEV), torch.zeros(4, 6, device=DEV),
                                workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def training_step(t, act):
    h, g, u = fp4.gated_gemm(t[0], t[1], t[2], act=act, save=True)
    return (h, g, u) + fp4.gated_gemm_backward(t[3], t[0], t[1], t[2], g, u, act=act)


def serving_step(x, b, sb, bg, sg, bu, su):
    q, s = fp4.int8_quantize(x)
    h = fp4.w8a8_gated_gemm(q, s, bg, sg, bu, su)
    q2, s2 = fp4.int8_quantize(h)
    return q, s, h, q2, s2, fp4.w8a8_gemm(q2, s2, b, sb)


def serving_inputs(m, n, k):
    g = gen(11)
    w = 1 / (73 * 73 * math.sqrt(k) * 0.03)
    return (torch.randn(m, k, generator=g, device=DEV).bfloat16(), codes(g, k, n), scales(g, k, w), codes(g, n, k),
            scales(g, n, w), codes(g, n, k), scales(g, n, w))


def test_repeats_are_bitwise_equal_and_other_streams_work():
    t, s = bf16_inputs(300, 520, 264, 10), serving_inputs(5, 1024, 512)
    first = training_step(t, "silu") + serving_step(*s)
    torch.cuda.synchronize(DEV)
    side = torch.cuda.Stream(device=DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        again = training_step(t, "silu") + serving_step(*s)
    side.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_captured_into_a_graph():
    t, s = bf16_inputs(130, 264, 136, 12), serving_inputs(3, 512, 256)

    def calls():
        return training_step(t, "gelu_tanh") + serving_step(*s)

    eager = [v.clone() for v in calls()]
    stream = torch.cuda.Stream(device=DEV)
    stream.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(stream):
        calls()
    torch.cuda.current_stream(DEV).wait_stream(stream)
    torch.cuda.synchronize(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = calls()
    for rep in range(4):
        for v in kept:
            v.fill_(1)
        graph.replay()
        torch.cuda.synchronize(DEV)
        for i, (a, b) in enumerate(zip(kept, eager)):
            assert torch.equal(a, b), f"replay {rep}: output {i}"
        fp4.gated_gemm(t[0], t[1], t[2])                 # eager work between the replays
        (t[0] * 2).sum()
        torch.cuda.synchronize(DEV)
