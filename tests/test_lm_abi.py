"""Host-side checks of the entry points of include/fp4g_lm.h: the library exports what the header declares and refuses
invalid arguments with the documented status before touching a device (no GPU needed: nothing here passes validation
with work to do)."""
import ctypes
import math
import os
import re

import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp4g_lm.h")

OK, EINVAL, EUNSUP, EALIGN = 0, 1, 2, 3
F32, BF16 = 0, 1
# Fake, aligned, non-overlapping "device" addresses: validation never dereferences them.
P = [0x10000000 * i for i in range(1, 16)]


@pytest.fixture(scope="module")
def lib():
    return fp4.lm._library()


def test_header_binding_and_library_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"^\s*fp4g_status\s+([a-z_0-9]+)\s*\(", text, re.M))
    assert declared == set(fp4.LM_SYMBOLS)
    for name in declared:
        assert hasattr(lib, name) and hasattr(fp4, name)


def norm(lib, rows=4, K=64, X=P[0], t=BF16, R=P[1], W=P[2], wt=BF16, eps=1e-6, H=P[3], Y=P[4]):
    return lib.rms_norm(rows, K, X, t, R, W, wt, eps, H, Y, None)


def quantize(lib, rows=4, K=64, X=P[0], t=BF16, R=P[1], W=P[2], wt=BF16, eps=1e-6, H=P[3], Y=P[4], c=P[5], ct=0, s=P[6]):
    return lib.rms_norm_quantize(rows, K, X, t, R, W, wt, eps, H, Y, c, ct, s, None)


@pytest.mark.parametrize("call", [norm, quantize])
def test_norm_refusals(lib, call):
    assert call(lib, rows=-1) == EINVAL and call(lib, K=-1) == EINVAL
    assert call(lib, rows=1 << 31) == EINVAL and call(lib, rows=1 << 30, K=1 << 30) == EINVAL
    assert call(lib, t=2) == EINVAL and call(lib, wt=2) == EINVAL and call(lib, wt=-1) == EINVAL
    for eps in (-1e-9, math.nan, math.inf):
        assert call(lib, eps=eps) == EINVAL
    assert call(lib, R=None) == EINVAL and call(lib, H=None) == EINVAL     # a sum without a residual, and the reverse
    assert call(lib, X=None) == EINVAL
    for name, base in (("X", P[0]), ("R", P[1]), ("W", P[2]), ("H", P[3]), ("Y", P[4])):
        assert call(lib, **{name: base + 1}) == EALIGN
        assert call(lib, t=F32, wt=F32, **{name: base + 2}) == EALIGN
    assert call(lib, Y=P[3]) == EINVAL                                     # Y and H the same
    assert call(lib, Y=P[0] + 128) == EINVAL and call(lib, H=P[1] + 128) == EINVAL   # over an input, but not in its place
    assert call(lib, Y=P[2]) == EINVAL and call(lib, H=P[2]) == EINVAL     # over the weight
    assert call(lib, Y=P[0], H=P[0]) == EINVAL
    assert call(lib, rows=0, X=None, Y=None) == OK


def test_norm_needs_its_results(lib):
    assert norm(lib, Y=None) == EINVAL
    assert quantize(lib, c=None) == EINVAL and quantize(lib, s=None) == EINVAL
    assert quantize(lib, ct=2) == EINVAL and quantize(lib, ct=-1) == EINVAL
    assert quantize(lib, s=P[6] + 2) == EALIGN
    assert quantize(lib, c=P[0]) == EINVAL and quantize(lib, s=P[5]) == EINVAL and quantize(lib, c=P[4]) == EINVAL
    assert norm(lib, K=0, X=None, W=None, R=None, H=None, Y=None) == OK


def backward(lib, rows=4, K=64, dY=P[0], X=P[1], t=BF16, W=P[2], wt=BF16, eps=1e-6, dH=P[3], dX=P[4], dW=P[5], w=P[6],
             wb=1 << 20):
    return lib.rms_norm_backward(rows, K, dY, X, t, W, wt, eps, dH, dX, dW, w, wb, None)


def test_norm_backward_refusals(lib):
    assert backward(lib, rows=-1) == EINVAL and backward(lib, K=1 << 31) == EINVAL
    assert backward(lib, rows=1 << 30, K=1 << 30) == EINVAL
    assert backward(lib, t=3) == EINVAL and backward(lib, wt=3) == EINVAL and backward(lib, eps=-1.0) == EINVAL
    assert backward(lib, W=None) == EINVAL                                 # the gradient of a weight that is not there
    for name in ("dY", "X", "dX", "w"):
        assert backward(lib, **{name: None}) == EINVAL
    for name, base in (("dY", P[0]), ("X", P[1]), ("W", P[2]), ("dH", P[3]), ("dX", P[4]), ("dW", P[5])):
        assert backward(lib, **{name: base + 1}) == EALIGN
    assert backward(lib, w=P[6] + 8) == EALIGN
    assert backward(lib, dX=P[1]) == EINVAL and backward(lib, dX=P[2]) == EINVAL     # over the rows, over the weight
    assert backward(lib, dX=P[0] + 64) == EINVAL and backward(lib, dW=P[4]) == EINVAL and backward(lib, w=P[1]) == EINVAL
    assert backward(lib, wb=16) == EINVAL
    assert backward(lib, w=P[0] - 16, wb=(1 << 64) - 16) == EINVAL         # reaches over the inputs
    assert backward(lib, rows=0, K=0, dY=None, X=None, dX=None) == OK
    n = ctypes.c_size_t(7)
    q = lib.rms_norm_backward_workspace_size
    assert q(-1, 4, BF16, ctypes.byref(n)) == EINVAL and q(4, 4, 2, ctypes.byref(n)) == EINVAL and q(4, 4, F32, None) == EINVAL
    assert q(0, 4, BF16, ctypes.byref(n)) == OK and n.value == 0
    assert q(4, 100, BF16, ctypes.byref(n)) == OK and n.value >= 400


def test_python_checks_come_before_the_library():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (fp4.rms_norm, fp4.rms_norm_quantize):
        with pytest.raises(ValueError, match="on a GPU"):
            call(x)
        with pytest.raises(TypeError, match="torch.Tensor"):
            call(None)
        with pytest.raises(TypeError, match="dtype"):
            call(x.half())
    with pytest.raises(TypeError, match="dtype"):
        fp4.rms_norm_backward(x, x.half())
    with pytest.raises(TypeError):
        fp4.rms_norm_backward_workspace_size(4, 4, torch.float16)


def test_binding_takes_every_argument_by_position():
    native = fp4.lm._binding()
    for name, count in (("rms_norm", 6), ("rms_norm_quantize", 7), ("rms_norm_backward", 7)):
        f = getattr(native, name)
        with pytest.raises(TypeError, match="expected"):
            f(*[None] * (count - 1))
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            f(*[None] * count)
