"""The root-mean-square norm against its formula in 64 bits: rows of every shape, both types, 8-bit codes, gradients.

Tolerances.  u = 2^-24 is fp32's half step, e that of the results' type (2^-24, or 2^-8 for bf16).
  Y    s is rounded once and two products follow: (3 u + e) |y|; 4 u covers the products of the errors.
  dX   s (g - n m) + dH with g = dY w: each of its three terms has at most 6 roundings, s^2 counted twice; m, the mean
       of g n, is a sum of chains of at most 48 additions (16 or 32 values a lane, 6 exchanges, 16 waves), each term
       with 2 roundings of its own: 8 u (|s g| + |s n m| + |dH|) + 52 u |s n| mean|g n| + e |dX|.  Rows of more than
       16384 bf16 (8192 fp32) elements have chains of K / 1024 + 22.
  dW   a sum of rows terms with 3 roundings each: (rows + 20) u sum|dY n| + e |dW|.
  The codes are compared with the same steps in fp32 and 64 bits, and have to be equal.
Below the smallest normal number, 2^-126, a step is 2^-149 (fp32) or 2^-133 (bf16): that much is added.
"""
import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: U}
TINY = {BF: 2.0 ** -133, F32: 2.0 ** -149}
EPS = 1e-6
SIZES = [(1, 1), (3, 7), (5, 64), (130, 128), (7, 129), (33, 500), (2, 1000), (9, 1117), (4, 2056), (3, 4096), (5, 8192),
         (2, 8201), (2, 16384), (1, 32768), (2, 40001)]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def inputs(rows, k, t, wt, residual, seed):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x = (r(rows, k) * (r(rows, 1) * 0.5).exp() * 3).to(t)
    w = None if wt is None else (1 + 0.3 * r(k)).to(wt)
    return x, w, (r(rows, k) * 2).to(t) if residual else None


def formula(x, w, res, eps=EPS):
    """h (in x's type), s and y in 64 bits."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    d = h.double()
    s = (d.square().mean(1, keepdim=True) + eps).rsqrt()
    return h, s, d * s * (1.0 if w is None else w.double())


def close(got, want, tol, what):
    err = (got.double() - want).abs()
    assert (err <= tol).all(), f"{what}: {(err - tol).max().item():.3g} past its tolerance, error {err.max().item():.3g}"


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("t,wt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF), (BF, None), (F32, None)])
@pytest.mark.parametrize("rows,k", SIZES)
def test_rows(rows, k, t, wt, residual):
    print(f"case rms_norm {rows}x{k} {t} weight {wt} residual {residual}", flush=True)
    x, w, res = inputs(rows, k, t, wt, residual, 1)
    out = fp4.rms_norm(x, w, eps=EPS, residual=res)
    y, h = out if residual else (out, x)
    torch.cuda.synchronize(DEV)
    ref_h, _, ref = formula(x, w, res)
    assert torch.equal(h, ref_h)
    close(y, ref, (4 * U + HALF[t]) * ref.abs() + TINY[t], "y")


def test_results_in_place_and_nothing_beyond():
    """Outputs in place of the inputs, rows that start anywhere, and what lies around them left as it was."""
    for t in (BF, F32):
        for rows, k in ((3, 129), (2, 4096), (2, 40001)):
            x, w, res = inputs(rows, k, t, t, True, 2)
            y, h = fp4.rms_norm(x, w, residual=res)
            for over in ("sum over residual", "sum over x", "both"):
                pad = [torch.full((rows * k + 66,), 7.0, dtype=t, device=DEV) for _ in range(2)]
                vx, vr = (p[33:33 + rows * k].view(rows, k) for p in pad)
                vx.copy_(x), vr.copy_(res)
                if over == "sum over residual":
                    gy, gh = fp4.rms_norm(vx, w, residual=vr, sum_out=vr)
                elif over == "sum over x":
                    gy, gh = fp4.rms_norm(vx, w, residual=vr, sum_out=vx)
                else:
                    gy, gh = fp4.rms_norm(vx, w, residual=vr, sum_out=vr, out=vx)
                torch.cuda.synchronize(DEV)
                assert torch.equal(gy, y) and torch.equal(gh, h), (t, rows, k, over)
                for p in pad:
                    assert (p[:33] == 7).all() and (p[33 + rows * k:] == 7).all()
            v = x.clone()
            assert fp4.rms_norm(v, w, out=v) is v and torch.equal(v, fp4.rms_norm(x, w))


def codes_of(x, w, res, kind, eps=EPS):
    """codes (as values), scales: the definition's steps, each 32-bit one in fp32."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    s = (1 / (h.double().square().mean(1, keepdim=True) + eps).sqrt()).float()
    y = h.float() * s
    if w is not None:
        y = y * w.float()
    top = 127.0 if kind == "int8" else 448.0
    most = y.abs().amax(1, keepdim=True)
    scale = most / torch.full_like(most, top)
    inv = (torch.ones_like(scale) / scale).clamp(max=torch.finfo(F32).max)
    bad = ~torch.isfinite(y).all(1, keepdim=True)
    q = torch.where(bad | (most == 0), torch.zeros_like(y), y * inv)
    q = q.round().clamp(-127, 127) if kind == "int8" else q.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    return q, torch.where(bad, torch.full_like(scale, float("nan")), scale)[:, 0], h


def values(codes):
    return codes.float() if codes.dtype == torch.int8 else codes.view(torch.float8_e4m3fn).float()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("t,wt,residual", [(BF, BF, True), (BF, F32, False), (F32, F32, True), (F32, BF, False), (BF, None, False)])
@pytest.mark.parametrize("rows,k", SIZES)
def test_codes(rows, k, t, wt, residual, kind):
    print(f"case rms_norm_quantize {rows}x{k} {t} weight {wt} residual {residual} {kind}", flush=True)
    x, w, res = inputs(rows, k, t, wt, residual, 3)
    codes, scales, *rest = fp4.rms_norm_quantize(x, w, eps=EPS, residual=res, codes=kind, keep=True)
    torch.cuda.synchronize(DEV)
    q, scale, h = codes_of(x, w, res, kind)
    assert torch.equal(values(codes), q) and torch.equal(scales, scale)
    if residual:
        assert torch.equal(rest[0], h)
    plain = fp4.rms_norm(x, w, eps=EPS, residual=res)
    assert torch.equal(rest[-1], plain[0] if residual else plain)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("k", [64, 2000, 40000])
def test_rows_without_finite_values_or_any(k, t, kind):
    """Zeros, infinities, NaN, the smallest and largest numbers; a neighbour's row is its own."""
    x, w, _ = inputs(9, k, t, t, False, 4)
    x[1] = 0
    x[2, k // 2] = float("inf")
    x[3, 0] = float("nan")
    x[4, k - 1] = float("-inf")
    x[5] = 1e-38
    x[6] = x[6].sign() * 3e37
    w[3 % k] = 0
    codes, scales, y = fp4.rms_norm_quantize(x, w, codes=kind, keep=True)
    torch.cuda.synchronize(DEV)
    q, scale, _ = codes_of(x, w, None, kind)
    assert torch.equal(values(codes), q) and torch.equal(scales.nan_to_num(-1), scale.nan_to_num(-1))
    assert scales[1] == 0 and not codes[1].any()
    for row in (2, 3, 4):
        assert torch.isnan(scales[row]) and not codes[row].any()
    assert torch.isfinite(y[[0, 1, 5, 6, 7, 8]].float()).all()
    # with eps == 0 a row of zeros has no norm
    y = fp4.rms_norm(x, w, eps=0.0)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0].float()).all()


def gradients(dy, h, w, dh, eps=EPS):
    """dX, dW in 64 bits and the sums of their terms' magnitudes."""
    d, g = h.double(), dy.double() * (1.0 if w is None else w.double())
    s = (d.square().mean(1, keepdim=True) + eps).rsqrt()
    n = d * s
    m = (g * n).mean(1, keepdim=True)
    dx = s * (g - n * m) + (0 if dh is None else dh.double())
    near = 8 * U * ((s * g).abs() + (s * n * m).abs() + (0 if dh is None else dh.double().abs()))
    chain = 52 if h.shape[1] <= (16384 if h.dtype == BF else 8192) else h.shape[1] / 1024 + 26
    near = near + chain * U * (s * n).abs() * (g * n).abs().mean(1, keepdim=True)
    t = dy.double() * n
    return dx, near, t.sum(0), (h.shape[0] + 20) * U * t.abs().sum(0)


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("t,wt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF), (BF, None), (F32, None)])
@pytest.mark.parametrize("rows,k", SIZES + [(2000, 128), (1100, 300), (700, 2048), (300, 8192), (70, 40001)])
def test_gradients(rows, k, t, wt, with_dh):
    print(f"case rms_norm_backward {rows}x{k} {t} weight {wt} dH {with_dh}", flush=True)
    x, w, dh = inputs(rows, k, t, wt, with_dh, 5)
    dy = torch.randn(rows, k, generator=gen(6), device=DEV).to(t)
    dx, dw = fp4.rms_norm_backward(dy, x, w, eps=EPS, dH=dh)
    torch.cuda.synchronize(DEV)
    rx, near, rw, near_w = gradients(dy, x, w, dh)
    close(dx, rx, near + (HALF[t] + U) * rx.abs() + TINY[t], "dX")
    assert (dw is None) == (w is None)
    if w is not None:
        close(dw, rw, near_w + (HALF[wt] + U) * rw.abs() + TINY[wt], "dW")


@pytest.mark.parametrize("scale", [2.0 ** 90, 2.0 ** -90])
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,k", [(3, 24), (40, 128), (9, 1117), (5, 8192), (2, 40001)])
def test_gradients_of_rows_whose_s_squared_leaves_the_range(rows, k, t, scale):
    """s is about 2^-90 or 2^90 and its square no fp32 number; every value of the formula is one."""
    print(f"case rms_norm_backward {rows}x{k} {t} scaled by {scale}", flush=True)
    x, w, _ = inputs(rows, k, t, t, False, 5)
    x = x * scale
    dy = torch.randn(rows, k, generator=gen(6), device=DEV).to(t)
    dx, dw = fp4.rms_norm_backward(dy, x, w, eps=0.0)
    torch.cuda.synchronize(DEV)
    rx, near, rw, near_w = gradients(dy, x, w, None, 0.0)
    close(dx, rx, near + (HALF[t] + U) * rx.abs() + TINY[t], "dX")
    close(dw, rw, near_w + (HALF[t] + U) * rw.abs() + TINY[t], "dW")


def test_gradients_agree_with_differences():
    """The slope of sum(Y dY) + sum(H dH) along random directions, by central differences of the formula in 64 bits: at
    a step of 1e-5 these are off by about 1e-10 of the slope's terms, the fp32 gradients by 1e-6 of them."""
    rows, k = 6, 200
    x, w, res = inputs(rows, k, F32, F32, True, 7)
    g = gen(8)
    dy, dh, vx, vw = (torch.randn(*s, generator=g, device=DEV) for s in ((rows, k), (rows, k), (rows, k), (k,)))
    h = x + res
    dx, dw = fp4.rms_norm_backward(dy, h, w, eps=EPS, dH=dh)

    def value(at):
        a = h.double() + at * vx.double()
        y = a * (a.square().mean(1, keepdim=True) + EPS).rsqrt() * (w.double() + at * vw.double())
        return (y * dy.double()).sum() + (a * dh.double()).sum()

    slope = (value(1e-5) - value(-1e-5)) / 2e-5
    terms = (dx.double() * vx.double()).abs().sum() + (dw.double() * vw.double()).abs().sum()
    got = (dx.double() * vx.double()).sum() + (dw.double() * vw.double()).sum()
    assert (got - slope).abs() <= 2e-6 * terms


def test_autograd_has_the_same_gradients():
    for t in (BF, F32):
        x, w, res = inputs(19, 136, t, t, True, 9)
        dy, dh = (torch.randn(19, 136, generator=gen(10 + i), device=DEV).to(t) for i in range(2))
        leaves = [v.clone().requires_grad_() for v in (x, w, res)]
        y, h = fp4.rms_norm(leaves[0], leaves[1], residual=leaves[2])
        assert y.requires_grad and h.requires_grad
        torch.autograd.backward([y, h], [dy, dh])
        dx, dw = fp4.rms_norm_backward(dy, h.detach(), w, dH=dh)
        assert torch.equal(leaves[0].grad, dx) and torch.equal(leaves[2].grad, dx) and torch.equal(leaves[1].grad, dw)
        assert leaves[0].grad.data_ptr() != leaves[2].grad.data_ptr()
        # the norm alone, the sum alone, and leaves that want nothing
        a = x.clone().requires_grad_()
        fp4.rms_norm(a, w).backward(dy)
        assert torch.equal(a.grad, fp4.rms_norm_backward(dy, x, w)[0])
        a = x.clone().requires_grad_()
        fp4.rms_norm(a, w, residual=res)[1].backward(dh)
        assert torch.equal(a.grad, dh)
        b = w.clone().requires_grad_()
        fp4.rms_norm(x, b).backward(dy.t().contiguous().t())
        assert torch.equal(b.grad, fp4.rms_norm_backward(dy, x, w)[1])
        a = x.clone().requires_grad_()
        fp4.rms_norm(a).sum().backward()
        assert a.grad is not None
        with torch.no_grad():
            assert not fp4.rms_norm(leaves[0], leaves[1]).requires_grad


def test_autograd_refuses_what_it_cannot_follow():
    x, w, res = inputs(4, 64, F32, F32, True, 11)
    a = x.clone().requires_grad_()
    (dx,) = torch.autograd.grad(fp4.rms_norm(a, w).square().sum(), a, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        dx.sum().backward()
    with pytest.raises(ValueError, match="recorded"):
        fp4.rms_norm(a, w, out=torch.empty_like(x))
    with pytest.raises(ValueError, match="no gradient"):
        fp4.rms_norm_quantize(a, w)
    with pytest.raises(ValueError, match="requires a gradient"):
        fp4.rms_norm(x, w, out=torch.empty_like(x).requires_grad_())
    # a row that a graph keeps and a later call overwrites
    y, h = fp4.rms_norm(a, w, residual=res)
    with torch.no_grad():
        fp4.rms_norm(x, w, residual=res, sum_out=h.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_workspaces_streams_and_captured_calls():
    """Forward, codes and gradients captured together and replayed among other work, against the eager results."""
    x, w, res = inputs(300, 1117, BF, BF, True, 12)
    dy = torch.randn(300, 1117, generator=gen(13), device=DEV).to(BF)
    size = fp4.rms_norm_backward_workspace_size(300, 1117)
    assert size > 0
    space = torch.full((size,), 255, dtype=torch.uint8, device=DEV)

    def calls():
        y, h = fp4.rms_norm(x, w, residual=res)
        q = fp4.rms_norm_quantize(x, w, residual=res, codes="e4m3")
        return (y, h, *q, *fp4.rms_norm_backward(dy, h, w, dH=dy, workspace=space))

    eager = [v.clone() for v in calls()]
    with pytest.raises(fp4.Fp4GemmError):
        fp4.rms_norm_backward(dy, x, w, workspace=space[:size - 16])
    side = torch.cuda.Stream(device=DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        for got, want in zip(calls(), eager):
            assert torch.equal(got, want)
    torch.cuda.synchronize(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for rep in range(4):
        for v in held:
            v.fill_(1)
        graph.replay()
        torch.cuda.synchronize(DEV)
        for got, want in zip(held, eager):
            assert torch.equal(got, want), rep
        fp4.rms_norm_backward(dy, x, w)
        torch.cuda.synchronize(DEV)


def test_no_rows_and_no_columns():
    for t in (BF, F32):
        none, w = torch.empty(0, 64, dtype=t, device=DEV), torch.ones(64, dtype=t, device=DEV)
        assert fp4.rms_norm(none, w).shape == (0, 64)
        assert fp4.rms_norm_quantize(none, w)[1].shape == (0,)
        dx, dw = fp4.rms_norm_backward(none, none, w)
        assert dx.shape == (0, 64) and not dw.any()
        flat = torch.empty(5, 0, dtype=t, device=DEV)
        assert fp4.rms_norm(flat).shape == (5, 0)
        assert not fp4.rms_norm_quantize(flat)[1].any()
        assert fp4.rms_norm_backward(flat, flat, w[:0])[1].shape == (0,)


def test_rows_past_32_bits():
    """2^31 + elements: the last rows come out as they do alone."""
    rows, k = 131080, 16384
    x = torch.empty(rows, k, dtype=BF, device=DEV)
    x.view(torch.int16)[:] = 0x3f80
    x[-3:] = torch.randn(3, k, generator=gen(14), device=DEV).to(BF)
    w = torch.randn(k, generator=gen(15), device=DEV).to(BF)
    codes, scales, y = fp4.rms_norm_quantize(x, w, keep=True)
    c, s, last = fp4.rms_norm_quantize(x[-3:].clone(), w, keep=True)
    assert torch.equal(y[-3:], last) and torch.equal(codes[-3:], c) and torch.equal(scales[-3:], s)
    del codes, y
    dx, dw = fp4.rms_norm_backward(x, x, w)
    d, _ = fp4.rms_norm_backward(x[-3:].clone(), x[-3:].clone(), w)
    torch.cuda.synchronize(DEV)
    assert torch.equal(dx[-3:], d) and torch.isfinite(dw.float()).all()


def test_more_rows_than_one_launch_holds():
    """2^27 + 3 rows of 8: sixteen lanes each, in two launches."""
    rows = (1 << 27) + 3
    x = torch.ones(rows, 8, dtype=BF, device=DEV)
    x[-5:] = torch.randn(5, 8, generator=gen(16), device=DEV).to(BF)
    y = fp4.rms_norm(x, eps=EPS)
    alone = fp4.rms_norm(x[-5:].clone(), eps=EPS)
    torch.cuda.synchronize(DEV)
    assert torch.equal(y[-5:], alone) and (y[:-5] == 1).all()
    del y
    codes, scales = fp4.rms_norm_quantize(x, eps=EPS)
    c, s = fp4.rms_norm_quantize(x[-5:].clone(), eps=EPS)
    torch.cuda.synchronize(DEV)
    assert torch.equal(codes[-5:], c) and torch.equal(scales[-5:], s) and (codes[:-5] == 127).all()
