"""Low-rank adapters beside a shared projection against the formula in 64 bits.

Tolerance.  u = 2^-24, e the half step of the results' type (2^-24 or 2^-8).  V = A x is a sum of K products in fp32, off by
(K + 8) u |A| |x|; scaling rounds it once; its bf16 terms keep it to 2^-8 each: two for bf16 results, three for fp32; the
second product adds up to 3 R terms in fp32, and D is rounded once, from a sum that may itself be rounded:
    |B| dV + (3 R + 8) u |B| |V| + u (|base| + |D|) + e |D|,   dV = (K + 8) u s |A| |x| + (2^-16 or 2^-24, + 2 u) |V|.
"""
import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: U}
SIZES = [  # M, N, K, R, L
    (1, 1, 8, 8, 1), (1, 4096, 4096, 16, 8), (3, 65, 72, 8, 2), (16, 129, 64, 24, 5), (17, 1000, 520, 16, 40), (64, 300, 1032, 64, 3),
    (100, 77, 136, 72, 100), (256, 513, 264, 128, 7), (257, 513, 264, 40, 7), (300, 1003, 2056, 256, 2), (1000, 130, 72, 16, 300),
    (2000, 2000, 520, 64, 4), (1500, 260, 64, 8, 1),
    (3000, 12000, 72, 40, 9), (2600, 13001, 64, 136, 3)]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def inputs(m, n, k, r, l, t, seed, order="random"):
    g = gen(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, a = rn(m, k).to(BF), (rn(l, r, k) / max(k, 1) ** 0.5).to(BF)
    b, base = (rn(l, n, r) * 0.5).to(BF), rn(m, n).to(t)
    if order == "random":
        index = torch.randint(-1, l, (m,), generator=g, device=DEV)
    elif order == "runs":
        index = (torch.arange(m, device=DEV) * 5 // m) % (l + 1) - 1
    else:
        index = torch.full((m,), l - 1, device=DEV)
    return base, x, a, b, index.int(), 0.5 + torch.rand(l, generator=g, device=DEV)


def formula(base, x, a, b, index, scales):
    m, k, r = x.shape[0], x.shape[1], a.shape[1]
    ref, tol = base.double(), U * base.double().abs()
    for i in range(a.shape[0]):
        at = torch.nonzero(index == i)[:, 0]
        if not at.numel():
            continue
        s = 1.0 if scales is None else scales[i].double()
        xd, ad, bd = x[at].double(), a[i].double(), b[i].double()
        v = xd @ ad.t() * s
        dv = (k + 8) * U * s * (xd.abs() @ ad.abs().t()) + ((2.0 ** -16 if base.dtype == BF else U) + 2 * U) * v.abs()
        ref[at] += v @ bd.t()
        tol[at] += dv @ bd.abs().t() + (3 * r + 8) * U * (v.abs() @ bd.abs().t())
    return ref, tol + (U + HALF[base.dtype]) * ref.abs() + 2.0 ** -133


def check(base, x, a, b, index, scales, **kw):
    d = fp4.adapter_gemm(base, x, a, b, index, scales=scales, **kw)
    torch.cuda.synchronize(DEV)
    ref, tol = formula(base, x, a, b, index, scales)
    err = (d.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} values past their tolerance, the worst by {(err - tol).max().item():.3g}"
    none = (index < 0) | (index >= a.shape[0])
    assert torch.equal(d[none], base[none])
    return d


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("order", ["random", "runs", "one"])
@pytest.mark.parametrize("m,n,k,r,l", SIZES)
def test_sizes(m, n, k, r, l, order, t):
    print(f"case adapter_gemm {m}x{n}x{k} r {r} of {l} {order} {t}", flush=True)
    base, x, a, b, index, scales = inputs(m, n, k, r, l, t, 1, order)
    check(base, x, a, b, index, scales)
    check(base, x, a, b, index, None)


@pytest.mark.parametrize("m", [5, 200, 700])
def test_in_place_and_nothing_beyond(m):
    n, k, r, l = 333, 136, 16, 6
    for t in (BF, F32):
        base, x, a, b, index, scales = inputs(m, n, k, r, l, t, 2)
        want = check(base, x, a, b, index, scales)
        pad = torch.full((m * n + 34,), 7.0, dtype=t, device=DEV)
        over = pad[17:17 + m * n].view(m, n)
        over.copy_(base)
        size = fp4.adapter_gemm_workspace_size(m, n, k, r, l)
        space = torch.full((size + 32,), 255, dtype=torch.uint8, device=DEV)
        d = fp4.adapter_gemm(over, x, a, b, index, scales=scales, out=over, workspace=space[:size])
        torch.cuda.synchronize(DEV)
        assert d is over and torch.equal(d, want)
        assert (pad[:17] == 7).all() and (pad[17 + m * n:] == 7).all() and (space[size:] == 255).all()
        with pytest.raises(fp4.Fp4GemmError):
            fp4.adapter_gemm(base, x, a, b, index, workspace=space[:size - 16])


@pytest.mark.parametrize("m", [40, 900])
def test_what_a_row_does_not_use_reaches_it_not(m):
    """NaN in rows without an adapter, in unused adapters, in another token of the same tile; indexes far outside."""
    n, k, r, l = 200, 72, 24, 5
    base, x, a, b, index, scales = inputs(m, n, k, r, l, F32, 3)
    index[index == 3] = 1
    index[0], index[1], index[2], index[m - 1] = -5, l, 2 ** 31 - 1, -(2 ** 31)
    want = check(base, x, a, b, index, scales)
    a[3], b[3], scales[3] = float("nan"), float("inf"), float("nan")
    x[(index < 0) | (index >= l)] = float("nan")
    assert torch.equal(fp4.adapter_gemm(base, x, a, b, index, scales=scales), want)
    x[10], index[10] = float("nan"), 1
    x[11, 3], index[11] = float("inf"), 1
    d = fp4.adapter_gemm(base, x, a, b, index, scales=scales)
    torch.cuda.synchronize(DEV)
    rest = torch.ones(m, dtype=torch.bool, device=DEV)
    rest[10:12] = False
    assert torch.isnan(d[10]).all() and not torch.isfinite(d[11]).any()
    assert torch.equal(d[rest], want[rest])


def test_tokens_by_the_thousand_and_adapters_by_the_thousand():
    m, n, k, r, l = 5000, 64, 64, 8, 8192
    base, x, a, b, index, scales = inputs(m, n, k, r, l, BF, 4)
    d = fp4.adapter_gemm(base, x, a, b, index, scales=scales)
    v = torch.einsum("mk,mrk->mr", x.double().cpu(), a.double().cpu()[index.long().clamp(min=0).cpu()])
    some = (index >= 0).cpu()[:, None]
    add = torch.einsum("mr,mnr->mn", v * scales.double().cpu()[index.long().clamp(min=0).cpu()][:, None],
                       b.double().cpu()[index.long().clamp(min=0).cpu()])
    ref = base.double().cpu() + torch.where(some, add, torch.zeros_like(add))
    torch.cuda.synchronize(DEV)
    assert ((d.double().cpu() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-3).all()


def test_a_row_is_the_same_in_any_company():
    """A token's result does not turn on the other tokens of the call, as long as K is cut the same way."""
    n, k, r, l = 300, 64, 16, 9
    base, x, a, b, index, scales = inputs(600, n, k, r, l, BF, 5)
    every = fp4.adapter_gemm(base, x, a, b, index, scales=scales)
    again = fp4.adapter_gemm(base, x, a, b, index, scales=scales)
    p = torch.randperm(600, generator=gen(6), device=DEV)
    mixed = fp4.adapter_gemm(base[p], x[p], a, b, index[p], scales=scales)
    few = fp4.adapter_gemm(base[:40], x[:40], a, b, index[:40], scales=scales)
    torch.cuda.synchronize(DEV)
    assert torch.equal(every, again) and torch.equal(every[p], mixed) and torch.equal(every[:40], few)


def test_captured_calls_and_other_streams():
    """Two graphs with workspaces of their own; the tokens' adapters change between replays."""
    for m in (48, 700):
        base, x, a, b, index, scales = inputs(m, 1000, 520, 16, 12, BF, 7)
        other = inputs(m, 1000, 520, 16, 12, BF, 8, "runs")[4]
        size = fp4.adapter_gemm_workspace_size(m, 1000, 520, 16, 12)
        live = index.clone()
        want = [fp4.adapter_gemm(base, x, a, b, i, scales=scales) for i in (index, other)]
        side = torch.cuda.Stream(device=DEV)
        side.wait_stream(torch.cuda.current_stream(DEV))
        with torch.cuda.stream(side):
            assert torch.equal(fp4.adapter_gemm(base, x, a, b, index, scales=scales), want[0])
        torch.cuda.synchronize(DEV)
        graphs, held = [], []
        for _ in range(2):
            space = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                held.append(fp4.adapter_gemm(base, x, a, b, live, scales=scales, workspace=space))
        for rep in range(4):
            live.copy_((index, other)[rep % 2])
            for d in held:
                d.fill_(1)
            for g in graphs:
                g.replay()
            torch.cuda.synchronize(DEV)
            assert all(torch.equal(d, want[rep % 2]) for d in held), rep
            fp4.adapter_gemm(base, x, a, b, index)
            torch.cuda.synchronize(DEV)


def test_empty_sizes():
    for m in (6, 300):
        base, x, a, b, index, scales = inputs(m, 40, 64, 8, 2, BF, 9)
        assert torch.equal(fp4.adapter_gemm(base, x, a[:0], b[:0], index), base)
        assert torch.equal(fp4.adapter_gemm(base, x, a[:, :0].contiguous(), b[:, :, :0].contiguous(), index), base)
        assert torch.equal(fp4.adapter_gemm(base, x[:, :0].contiguous(), a[:, :, :0].contiguous(), b, index), base)
        assert fp4.adapter_gemm(base[:, :0].contiguous(), x, a, b[:, :0].contiguous(), index).shape == (m, 0)
    assert fp4.adapter_gemm(base[:0], x[:0], a, b, index[:0]).shape == (0, 40)


def test_adapters_and_rows_past_32_bits():
    """The last of 2^31 + elements of B, and of base."""
    l, n, r = 1100, 8192, 256
    b = torch.zeros(l, n, r, dtype=BF, device=DEV)
    b[-1] = torch.randn(n, r, generator=gen(10), device=DEV).to(BF)
    a, x = (torch.randn(l, r, 8, generator=gen(11), device=DEV).to(BF), torch.randn(3, 8, generator=gen(12), device=DEV).to(BF))
    base = torch.zeros(3, n, dtype=F32, device=DEV)
    index = torch.tensor([l - 1, 0, l - 1], dtype=torch.int32, device=DEV)
    d = fp4.adapter_gemm(base, x, a, b, index)
    alone = fp4.adapter_gemm(base, x, a[-1:].clone(), b[-1:].clone(), torch.zeros_like(index))
    torch.cuda.synchronize(DEV)
    assert torch.equal(d[[0, 2]], alone[[0, 2]]) and not d[1].any()
    del b
    m, n = 70000, 32768
    base = torch.zeros(m, n, dtype=BF, device=DEV)
    x, a, b = (torch.randn(*s, generator=gen(13 + i), device=DEV).to(BF) for i, s in enumerate(((m, 8), (2, 8, 8), (2, n, 8))))
    index = torch.full((m,), -1, dtype=torch.int32, device=DEV)
    index[-2:] = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    last = fp4.adapter_gemm(base[-2:].clone(), x[-2:].clone(), a, b, index[-2:].clone())
    d = fp4.adapter_gemm(base, x, a, b, index, out=base)
    torch.cuda.synchronize(DEV)
    assert torch.equal(d[-2:], last) and not d[:-2].any()


def test_no_gradient_is_lost():
    base, x, a, b, index, scales = inputs(4, 16, 8, 8, 2, BF, 16)
    for i in range(4):
        leaves = [v.clone() for v in (base, x, a, b)]
        leaves[i].requires_grad_()
        with pytest.raises(ValueError, match="no gradient"):
            fp4.adapter_gemm(*leaves, index)
        with torch.no_grad():
            assert not fp4.adapter_gemm(*leaves, index).requires_grad
