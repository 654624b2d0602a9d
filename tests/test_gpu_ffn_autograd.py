"""gated_gemm under autograd: what a graph records is what gated_gemm_backward gives, and nothing is lost in silence."""
import importlib.util
import os

import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4
from tests.test_gpu_ffn import ACTS, DEV, bf16_inputs, gen

pytestmark = pytest.mark.gpu


def leaves(m, n, k, wanted=(True, True, True)):
    *t, dh = bf16_inputs(m, n, k, 61)
    return [v.requires_grad_(w) for v, w in zip(t, wanted)], dh


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 1, 8), (3, 65, 72), (130, 257, 136)])
def test_a_recorded_call_has_its_gradients(m, n, k, act):
    print(f"case gated_gemm under autograd {m}x{n}x{k} {act}", flush=True)
    t, dh = leaves(m, n, k)
    with torch.no_grad():
        h, g, u = fp4.gated_gemm(*t, act=act, save=True)
        want = fp4.gated_gemm_backward(dh, *t, g, u, act=act)
    got = fp4.gated_gemm(*t, act=act)
    assert not h.requires_grad and got.requires_grad and torch.equal(got.detach(), h)
    got.backward(dh)
    torch.cuda.synchronize(DEV)
    for leaf, w in zip(t, want):
        assert torch.equal(leaf.grad, w)


def test_a_residual_keeps_both_of_its_gradients():
    t, dh = leaves(17, 72, 72)
    (dx,) = torch.autograd.grad(t[0] + fp4.gated_gemm(*t), t[:1], dh)
    (through,) = torch.autograd.grad(fp4.gated_gemm(*t), t[:1], dh)
    torch.cuda.synchronize(DEV)
    assert through.any() and torch.equal(dx, dh + through)


@pytest.mark.parametrize("wanted", [(True, False, False), (False, True, False), (False, False, True), (True, False, True)])
def test_leaves_that_ask_for_none_get_none(wanted):
    t, dh = leaves(5, 40, 64, wanted)
    every, _ = leaves(5, 40, 64)
    fp4.gated_gemm(*t).backward(dh)
    fp4.gated_gemm(*every).backward(dh)
    torch.cuda.synchronize(DEV)
    for leaf, other, w in zip(t, every, wanted):
        assert torch.equal(leaf.grad, other.grad) if w else leaf.grad is None


def test_kept_products_results_in_place_and_no_grad():
    t, dh = leaves(9, 48, 40)
    with torch.no_grad():
        plain, g, u = fp4.gated_gemm(*t, save=True)
    h, kg, ku = fp4.gated_gemm(*t, save=True)
    assert h.requires_grad and not kg.requires_grad and not ku.requires_grad
    assert torch.equal(kg, g) and torch.equal(ku, u)
    out = torch.empty_like(plain)
    h = fp4.gated_gemm(*t, out=out)
    assert h is out and torch.equal(out.detach(), plain)
    (dx,) = torch.autograd.grad(h, t[:1], dh)
    (want,) = torch.autograd.grad(fp4.gated_gemm(*t), t[:1], dh)
    torch.cuda.synchronize(DEV)
    assert torch.equal(dx, want)
    with torch.inference_mode():
        assert not fp4.gated_gemm(*t).requires_grad
    assert not fp4.gated_gemm(*(v.detach() for v in t)).requires_grad


def test_second_derivatives_are_refused():
    """Also where nothing but the inputs carries them (the incoming gradient is a constant) and other terms are there."""
    t, _ = leaves(4, 16, 24)
    (dx,) = torch.autograd.grad(fp4.gated_gemm(*t).float().sum(), t[:1], create_graph=True)
    (plain,) = torch.autograd.grad(fp4.gated_gemm(*t).float().sum(), t[:1])
    assert torch.equal(dx.detach(), plain)              # first derivatives are there all the same
    with pytest.raises(RuntimeError, match="second derivatives"):
        (dx.float().square().sum() + t[0].float().sum()).backward()


def test_refusals_are_those_of_the_plain_call():
    t, _ = leaves(4, 16, 24)
    with pytest.raises(ValueError, match="act"):
        fp4.gated_gemm(*t, act="relu")
    with pytest.raises(TypeError, match="dtype"):
        fp4.gated_gemm(t[0], t[1].float(), t[2])
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        fp4.gated_gemm(t[0], None, t[2])


def test_the_example_hands_on_what_autograd_asks_for():
    """Leading dimensions, a frozen weight, and second derivatives that raise rather than vanish."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward_example_again", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    t, dh = leaves(6, 16, 24, (True, True, False))
    h = example.gated_product(t[0].reshape(2, 3, 24), *t[1:])
    h.backward(dh.reshape(2, 3, 16), retain_graph=True)
    torch.cuda.synchronize(DEV)
    assert t[0].grad.any() and t[1].grad.any() and t[2].grad is None
    (dx,) = torch.autograd.grad(h.float().sum(), t[:1], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        (dx.float().square().sum() + t[0].float().sum()).backward()


@pytest.mark.parametrize("m,n", [(5, 33), (130, 257), (40, 64)])
def test_gradients_that_start_at_any_element(m, n):
    """Row slices of tensors with odd rows start inside a 16-byte line."""
    print(f"case gated_gemm_backward of slices {m}x{n}", flush=True)
    t, _ = leaves(m, n, 72, (False,) * 3)
    dh = torch.randn(m * n + 8, generator=gen(62), device=DEV).bfloat16()
    kept = torch.randn(2, m * n + 8, generator=gen(63), device=DEV)
    for first in (1, 3, 7):
        d, g, u = dh[first:first + m * n].view(m, n), *(v[first:first + m * n].view(m, n) for v in kept)
        got = fp4.gated_gemm_backward(d, *t, g, u)
        want = fp4.gated_gemm_backward(d.clone(), *t, g.clone(), u.clone())
        torch.cuda.synchronize(DEV)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    rows, _ = leaves(m - 1, n, 72)
    h = fp4.gated_gemm(*rows)
    h.backward(dh[:m * n].view(m, n)[1:])                # as a backward pass hands it over
    torch.cuda.synchronize(DEV)
    assert rows[0].grad.any()
