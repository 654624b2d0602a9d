"""The feed-forward example: the operators together, as a program uses them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("feed_forward_example", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def reference(x, wg, wu, wd, act):
    f = torch.nn.functional
    act = {"silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[act]
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    return (act(x @ wg.t()) * (x @ wu.t())) @ wd.t()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("shape", [(1,), (5,), (2, 3), (130,)])
def test_int8_block(example, shape, act):
    """Codes are off by half a step of max|x| / 127.  Normal rows of 512 and 1024 have a maximum of
    about 3.3 standard deviations, so an operand's relative error is 3.3 / 127 / sqrt(12) = 0.0075;
    weights, activations and the hidden rows (whose products have heavier tails: three times that)
    add to less than 0.05."""
    print(f"case int8 block {shape} {act}", flush=True)
    wg, wu, wd = example.weights(1024, 512, DEV)
    x = torch.randn(*shape, 512, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).bfloat16()
    y = example.Int8FeedForward(wg, wu, wd, act)(x)
    torch.cuda.synchronize(DEV)
    want = reference(x.reshape(-1, 512), wg, wu, wd, act).reshape(*shape, 512)
    assert y.shape == want.shape and y.dtype is torch.bfloat16
    assert ((y.double() - want).norm() / want.norm()).item() < 0.05


def test_gradients_reach_every_leaf(example):
    """Against autograd through the 64-bit formula.  The kernels round dG and dU, the incoming
    gradient and the results to bf16, each at most 2^-8 of its value, and sums of such terms
    relative to the whole gradient no more than their total: 4 * 2^-8."""
    wg, wu, _ = example.weights(96, 64, DEV)
    x = torch.randn(3, 17, 64, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV).bfloat16()
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu)]
    h = example.gated_product(*leaves)
    assert h.shape == (3, 17, 96)
    h.float().square().sum().backward()
    torch.cuda.synchronize(DEV)
    wide = [t.double().requires_grad_() for t in (x, wg, wu)]
    hw = torch.nn.functional.silu(wide[0] @ wide[1].t()) * (wide[0] @ wide[2].t())
    hw.square().sum().backward()
    for a, b in zip(leaves, wide):
        assert a.grad.shape == b.grad.shape
        assert ((a.grad.double() - b.grad).norm() / b.grad.norm()).item() < 4 * 2.0 ** -8
    # an incoming gradient that is a broadcast of one value is made contiguous on the way
    (d,) = torch.autograd.grad(example.gated_product(*leaves).sum(), leaves[:1])
    assert torch.isfinite(d).all()


def test_training_goes_down(example):
    losses = example.train(12, 200, 272, 128)
    assert losses[-1] < 0.7 * losses[0]
