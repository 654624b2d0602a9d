"""The operators around a model's products in the order in which a model uses them, and its example."""
import importlib.util
import os

import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U, B = 2.0 ** -24, 2.0 ** -8


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "language_model.py")
    spec = importlib.util.spec_from_file_location("example_language_model", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


@pytest.mark.parametrize("m", [1, 30, 300])
def test_norm_into_int8_and_w4a8_products(m):
    """The codes are what w8a8_gemm and w4a8_gemm take: their products are those of the values the codes stand for."""
    k, n = 512, 200
    x, res, w = rn(1, m, k).bfloat16(), rn(2, m, k).bfloat16(), (1 + 0.1 * rn(3, k)).bfloat16()
    codes, scales, h = fp4.rms_norm_quantize(x, w, residual=res)
    bq, bs = fp4.int8_quantize(rn(4, n, k))
    d = fp4.w8a8_gemm(codes, scales, bq, bs, out_dtype=torch.float32)
    # whole sums, exact in 64 bits; of scaled values 64 bits would lose what is left where they cancel
    ref = codes.double() @ bq.double().t() * scales.double()[:, None] * bs.double()
    torch.cuda.synchronize(DEV)
    assert ((d.double() - ref).abs() <= 4 * U * ref.abs() + 1e-30).all()     # the sum is exact, two products follow
    y = fp4.rms_norm(x, w, residual=res)[0].double()
    step = scales.double()[:, None] * 0.5 * (1 + 2.0 ** -20) + (B + 4 * U) * y.abs()
    assert ((codes.double() * scales.double()[:, None] - y).abs() <= step).all()
    codes, scales, h2 = fp4.rms_norm_quantize(x, w, residual=res, codes="e4m3")
    assert torch.equal(h, h2)
    nibbles = torch.randint(0, 256, (n, k // 2), generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).to(torch.uint8)
    sb = (0.01 + 0.04 * torch.rand(n, k // 128, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV)).bfloat16()
    d = fp4.w4a8_gemm(codes, scales, nibbles, sb, out_dtype=torch.float32)
    both = torch.stack((nibbles & 15, nibbles >> 4), 2).reshape(n, k).to(torch.int64)
    q = torch.where(both > 7, both - 16, both).double() * sb.double().repeat_interleave(128, 1)
    a = codes.view(torch.float8_e4m3fn).double() * scales.double()[:, None]
    torch.cuda.synchronize(DEV)
    assert ((d.double() - a @ q.t()).abs() <= (k + 16) * U * (a.abs() @ q.abs().t())).all()


def test_served_block_with_adapters():
    """Rows without an adapter are the block's own, in place; the others differ by what adapter_gemm adds."""
    ex = example()
    m, k, n = 70, 256, 512
    p = ex.parameters(k, n, 64, DEV)
    adapters = ((rn(7, 5, 16, n) / n ** 0.5).bfloat16(), (rn(8, 5, k, 16) / 4).bfloat16(), torch.rand(5, device=DEV) + 0.5)
    x, res = rn(9, m, k).bfloat16(), rn(10, m, k).bfloat16()
    index = (torch.arange(m, device=DEV) % 6 - 1).int()
    block = ex.ServedBlock(p[0], *p[1:4], adapters)
    y, total = block(x, res, index)
    bare, _ = block(x, res, torch.full_like(index, -1))
    codes, scales, total2, rows = fp4.rms_norm_quantize(x, p[0], residual=res, keep=True)
    h = fp4.w8a8_gated_gemm(codes, scales, *block.gate, *block.up, act="silu")
    want = fp4.adapter_gemm(bare, h, *adapters[:2], index, scales=adapters[2])
    torch.cuda.synchronize(DEV)
    assert torch.equal(y, want) and torch.equal(total, total2) and torch.equal(y[index < 0], bare[index < 0])
    assert not torch.equal(y, bare)


def step_by_hand(x, p, target):
    """The example's loss and gradients through the explicit functions; its torch product by the rules of bf16 autograd."""
    norm1, wg, wu, wd, norm2, head = p
    n1 = fp4.rms_norm(x, norm1)
    h, g, u = fp4.gated_gemm(n1, wg, wu, save=True)
    d = h @ wd.t()
    y, s = fp4.rms_norm(d, norm2, residual=x)
    loss, lse = fp4.cross_entropy_gemm(y, head, target, save=True)
    some = (target != -100).sum()
    dl = torch.full_like(loss, 1.0) / some
    dy, dhead = fp4.cross_entropy_gemm_backward(dl, y, head, target, lse)
    dd, dnorm2 = fp4.rms_norm_backward(dy, s, norm2)
    dh, dwd = dd @ wd, dd.t() @ h
    dn1, dwg, dwu = fp4.gated_gemm_backward(dh, n1, wg, wu, g, u)
    _, dnorm1 = fp4.rms_norm_backward(dn1, x, norm1)
    return loss.sum() / some, (dnorm1, dwg, dwu, dwd, dnorm2, dhead)


@pytest.mark.parametrize("m", [9, 200])
def test_a_training_step_by_autograd_and_by_hand(m):
    ex = example()
    k, n, v = 128, 264, 515
    p = ex.parameters(k, n, v, DEV, seed=4)
    x = rn(11, m, k).bfloat16()
    target = torch.randint(0, v, (m,), generator=torch.Generator(device=DEV).manual_seed(12), device=DEV)
    target[: m // 3] = -100
    loss, grads = step_by_hand(x, p, target)
    leaves = [t.clone().requires_grad_() for t in p]
    got = ex.loss_of(x, leaves, target)
    d = torch.autograd.grad(got, leaves)
    torch.cuda.synchronize(DEV)
    assert torch.equal(got.detach(), loss)
    for a, b, name in zip(d, grads, ("norm1", "wg", "wu", "wd", "norm2", "head")):
        assert torch.equal(a, b), name
        assert a.isfinite().all() and a.any(), name


def test_a_training_step_against_64_bits():
    """The whole step's gradients against autograd in 64 bits from the same parameters: each of the step's five bf16
    results on the way is off by half a step (2^-8), so the relative error of a gradient's norm stays below 6 half steps."""
    ex = example()
    m, k, n, v = 96, 128, 256, 400
    p = ex.parameters(k, n, v, DEV, seed=5)
    x = rn(13, m, k).bfloat16()
    target = torch.randint(0, v, (m,), generator=torch.Generator(device=DEV).manual_seed(14), device=DEV)
    target[5:20] = -100
    _, grads = step_by_hand(x, p, target)
    q = [t.double().requires_grad_() for t in p]
    rms = lambda t, w: t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w  # noqa: E731
    xd = x.double()
    a = rms(xd, q[0])
    h = torch.nn.functional.silu(a @ q[1].t()) * (a @ q[2].t())
    y = rms(h @ q[3].t() + xd, q[4])
    loss = torch.nn.functional.cross_entropy(y @ q[5].t(), target, ignore_index=-100)
    for d, r, name in zip(grads, torch.autograd.grad(loss, q), ("norm1", "wg", "wu", "wd", "norm2", "head")):
        assert (d.double() - r).norm() <= 6 * B * r.norm(), name


def test_a_captured_training_step():
    """The explicit functions of a whole step in one graph, replayed on other tokens between eager steps."""
    ex = example()
    m, k, n, v = 130, 128, 264, 515
    p = ex.parameters(k, n, v, DEV, seed=6)
    xs = [rn(20 + i, m, k).bfloat16() for i in range(3)]
    ts = [torch.randint(0, v, (m,), generator=torch.Generator(device=DEV).manual_seed(30 + i), device=DEV) for i in range(3)]
    for i, t in enumerate(ts):
        t[: 40 * i] = -100

    def step(x, target):
        y, s = fp4.rms_norm(x, p[4], residual=x)
        loss, lse = fp4.cross_entropy_gemm(y, p[5], target, save=True)
        dy, dhead = fp4.cross_entropy_gemm_backward(torch.ones_like(loss), y, p[5], target, lse)
        return loss, dhead, *fp4.rms_norm_backward(dy, s, p[4], dH=dy)

    want = [[r.clone() for r in step(x, t)] for x, t in zip(xs, ts)]
    live_x, live_t = xs[0].clone(), ts[0].clone()
    side = torch.cuda.Stream(device=DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        step(live_x, live_t)
    torch.cuda.current_stream(DEV).wait_stream(side)
    torch.cuda.synchronize(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(live_x, live_t)
    for rep in range(5):
        live_x.copy_(xs[rep % 3]), live_t.copy_(ts[rep % 3])
        graph.replay()
        torch.cuda.synchronize(DEV)
        for a, b in zip(held, want[rep % 3]):
            assert torch.equal(a, b), rep
        step(xs[1], ts[2])
        torch.cuda.synchronize(DEV)


def test_calls_from_several_threads():
    """Each thread on its own stream; results are those of one call after the other."""
    import threading
    x, res, w = rn(40, 200, 520).bfloat16(), rn(41, 200, 520).bfloat16(), rn(42, 520).bfloat16()
    head = (rn(43, 700, 520) / 23).bfloat16()
    t = torch.arange(200, device=DEV) * 3
    a, b, base = (rn(44, 4, 16, 520) / 23).bfloat16(), rn(45, 4, 300, 16).bfloat16(), rn(46, 200, 300)
    index = (torch.arange(200, device=DEV) % 5 - 1).int()

    def calls():
        y, h = fp4.rms_norm(x, w, residual=res)
        loss, lse = fp4.cross_entropy_gemm(y, head, t, save=True)
        return (y, h, loss, *fp4.cross_entropy_gemm_backward(loss, y, head, t, lse), fp4.adapter_gemm(base, y, a, b, index),
                *fp4.rms_norm_backward(y, h, w))

    want = calls()
    torch.cuda.synchronize(DEV)
    got, errors = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream(device=DEV)
            with torch.cuda.stream(s):
                for _ in range(4):
                    got[i] = calls()
            s.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    for r in got:
        assert all(torch.equal(p, q) for p, q in zip(r, want))


def test_the_example_runs():
    losses = example().train(3, 64, 128, 256, 300)
    assert len(losses) == 3 and all(v == v and abs(v) < 1e4 for v in losses)
