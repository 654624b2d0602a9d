"""More rows of a norm than one launch holds: the rows of the second come out as they do alone."""
import ctypes

import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4
from tests.ffn_plans import internal

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
LAST = 5


def limit(rows, k):
    """Rows of one launch, as the library cuts them."""
    f = internal("_ZN4fp4g20rms_norm_launch_rowsEllb", ctypes.c_int64, 2)
    f.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_bool]
    return f(rows, k, True)


@pytest.fixture(params=[1, 8])
def rows_of(request):
    """Rows of 1 and of 8 elements, those of the first launch alike (their sum with the residual is 2), the last at random."""
    k = request.param
    rows = limit(1 << 30, k) + LAST - 2
    assert limit(rows, k) == rows - LAST + 2 and rows < 1 << 30          # two launches, the second of three rows
    print(f"case rms_norm {rows}x{k}", flush=True)
    torch.cuda.empty_cache()
    g = torch.Generator(device=DEV).manual_seed(k)
    x = torch.full((rows, k), 0.5, dtype=BF, device=DEV)
    res = torch.full((rows, k), 1.5, dtype=BF, device=DEV)
    for t in (x, res):
        t[-LAST:] = torch.randn(LAST, k, generator=g, device=DEV).to(BF)
    w = (1 + torch.rand(k, generator=g, device=DEV)).to(BF)
    yield x, res, w
    torch.cuda.synchronize(DEV)
    torch.cuda.empty_cache()


def same(got, alone, first):
    assert torch.equal(got[-LAST:], alone[-LAST:])
    assert (got[:-LAST] == first[0]).all()


def test_rows_and_sums(rows_of):
    x, res, w = rows_of
    two = [t[-LAST - 1:].clone() for t in (x, res)]              # a row of the many, and the last
    y, h = fp4.rms_norm(x, w, residual=res)
    a, b = fp4.rms_norm(two[0], w, residual=two[1])
    same(y, a, a)
    same(h, b, b)
    # without a residual, in place
    a = fp4.rms_norm(two[0], w)
    assert fp4.rms_norm(x, w, out=x) is x
    same(x, a, a)


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_codes_and_scales(rows_of, codes):
    x, res, w = rows_of
    two = [t[-LAST - 1:].clone() for t in (x, res)]
    many = fp4.rms_norm_quantize(x, w, residual=res, codes=codes, keep=True)
    few = fp4.rms_norm_quantize(two[0], w, residual=two[1], codes=codes, keep=True)
    for got, alone in zip(many, few):
        same(got, alone, alone)


def test_gradients(rows_of):
    """Of as many rows: one launch, whose workgroups walk them."""
    x, dy, w = rows_of
    dx, dw = fp4.rms_norm_backward(dy, x, w)
    alone, _ = fp4.rms_norm_backward(dy[-LAST - 1:].clone(), x[-LAST - 1:].clone(), w)
    same(dx, alone, alone)
    assert torch.isfinite(dw.float()).all()
