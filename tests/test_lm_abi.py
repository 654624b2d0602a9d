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


def loss(lib, M=4, V=50, K=64, X=P[0], W=P[1], t=P[2], out=P[3], lse=P[4], w=P[5], wb=1 << 24):
    return lib.cross_entropy_gemm(M, V, K, X, W, t, -100, out, lse, w, wb, None)


def loss_grad(lib, M=4, V=50, K=64, dL=P[6], X=P[0], W=P[1], t=P[2], lse=P[4], dX=P[7], dW=P[8], w=P[5], wb=1 << 24):
    return lib.cross_entropy_gemm_backward(M, V, K, dL, X, W, t, -100, lse, dX, dW, w, wb, None)


@pytest.mark.parametrize("call", [loss, loss_grad])
def test_loss_refusals(lib, call):
    for name in ("M", "V", "K"):
        assert call(lib, **{name: -1}) == EINVAL and call(lib, **{name: 1 << 31}) == EINVAL
    assert call(lib, V=0) == EINVAL                      # rows, and no vocabulary
    assert call(lib, K=12) == EUNSUP and call(lib, K=(1 << 21) + 8) == EUNSUP and call(lib, M=(1 << 25) + 1, V=8) == EUNSUP
    assert call(lib, V=1 << 30, K=1 << 21) == EINVAL
    for name in ("X", "W", "t", "w"):
        assert call(lib, **{name: None}) == EINVAL
    for name, base, by in (("X", P[0], 8), ("W", P[1], 8), ("t", P[2], 4), ("lse", P[4], 2), ("w", P[5], 8)):
        assert call(lib, **{name: base + by}) == EALIGN
    assert call(lib, wb=64) == EINVAL
    assert call(lib, w=P[0] - 16, wb=(1 << 64) - 16) == EINVAL
    assert call(lib, w=P[1]) == EINVAL


def test_loss_results_are_checked(lib):
    assert loss(lib, out=None) == EINVAL and loss(lib, out=P[3] + 1) == EALIGN
    assert loss(lib, out=P[2]) == EINVAL and loss(lib, lse=P[3]) == EINVAL
    assert loss(lib, M=0, X=None, t=None, out=None) == OK
    assert loss_grad(lib, dL=None) == EINVAL and loss_grad(lib, lse=None) == EINVAL
    assert loss_grad(lib, dX=P[7] + 8) == EALIGN and loss_grad(lib, dW=P[8] + 8) == EALIGN
    assert loss_grad(lib, dX=P[0]) == EINVAL and loss_grad(lib, dW=P[1]) == EINVAL and loss_grad(lib, dW=P[7]) == EINVAL
    assert loss_grad(lib, dX=None, dW=None) == OK        # nothing is wanted
    assert loss_grad(lib, K=0) == OK


def test_loss_workspace_queries(lib):
    n, least = ctypes.c_size_t(7), ctypes.c_size_t(7)
    f, b = lib.cross_entropy_gemm_workspace_size, lib.cross_entropy_gemm_backward_workspace_size
    assert f(-1, 4, 64, ctypes.byref(n)) == EINVAL and f(4, 4, 20, ctypes.byref(n)) == EUNSUP and f(4, 4, 64, None) == EINVAL
    assert b(4, 0, 64, ctypes.byref(n), ctypes.byref(least)) == EINVAL and b(4, 4, 64, ctypes.byref(n), None) == EINVAL
    assert f(0, 4, 64, ctypes.byref(n)) == OK and n.value == 0
    assert b(0, 4, 64, ctypes.byref(n), ctypes.byref(least)) == OK and n.value == 0 and least.value == 0
    for m, v, k in ((1, 1, 8), (301, 1003, 520), (8192, 131072, 4096), (3, 1 << 30, 64), (1 << 25, 1000, 64)):
        assert f(m, v, k, ctypes.byref(n)) == OK and n.value >= 2 * m * k
        assert b(m, v, k, ctypes.byref(n), ctypes.byref(least)) == OK and 0 < least.value <= n.value
    # a step of 8192 tokens over 131072: far less than its logits (4 GB in fp32)
    assert b(8192, 131072, 4096, ctypes.byref(n), ctypes.byref(least)) == OK and n.value < 1 << 29


def adapters(lib, M=4, N=40, K=64, R=16, L=3, base=P[0], X=P[1], A=P[2], B=P[3], s=P[4], i=P[5], D=P[6], t=BF16, w=P[7],
             wb=1 << 20):
    return lib.adapter_gemm(M, N, K, R, L, base, X, A, B, s, i, D, t, w, wb, None)


def test_adapter_refusals(lib):
    for name in ("M", "N", "K", "R", "L"):
        assert adapters(lib, **{name: -1}) == EINVAL and adapters(lib, **{name: 1 << 31}) == EINVAL
    assert adapters(lib, K=12) == EUNSUP and adapters(lib, R=12) == EUNSUP and adapters(lib, R=264) == EUNSUP
    assert adapters(lib, L=8193) == EUNSUP and adapters(lib, K=(1 << 21) + 8) == EUNSUP
    assert adapters(lib, M=(1 << 25) + 1) == EUNSUP and adapters(lib, N=(1 << 30) + 1) == EUNSUP
    assert adapters(lib, N=1 << 30, R=256, L=8192) == EINVAL               # more than 2^50 elements
    assert adapters(lib, t=2) == EINVAL
    for name in ("base", "X", "A", "B", "i", "D", "w"):
        assert adapters(lib, **{name: None}) == EINVAL
    for name, at, by in (("base", P[0], 1), ("X", P[1], 8), ("A", P[2], 8), ("B", P[3], 8), ("s", P[4], 2), ("i", P[5], 2),
                         ("D", P[6], 1), ("w", P[7], 8)):
        assert adapters(lib, **{name: at + by}) == EALIGN
    assert adapters(lib, D=P[0] + 64) == EINVAL and adapters(lib, D=P[1]) == EINVAL and adapters(lib, D=P[3]) == EINVAL
    assert adapters(lib, w=P[0]) == EINVAL and adapters(lib, w=P[6]) == EINVAL
    assert adapters(lib, wb=64) == EINVAL and adapters(lib, w=P[0] - 16, wb=(1 << 64) - 16) == EINVAL
    assert adapters(lib, M=0, base=None, X=None, i=None, D=None) == OK and adapters(lib, N=0, base=None, B=None, D=None) == OK
    n = ctypes.c_size_t(7)
    q = lib.adapter_gemm_workspace_size
    assert q(-1, 4, 64, 8, 1, ctypes.byref(n)) == EINVAL and q(4, 4, 20, 8, 1, ctypes.byref(n)) == EUNSUP
    assert q(4, 4, 64, 8, 1, None) == EINVAL
    assert q(0, 4, 64, 8, 1, ctypes.byref(n)) == OK and n.value == 0
    assert q(4, 4, 64, 8, 1, ctypes.byref(n)) == OK and n.value >= 4 * 8 * 4


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
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="on a GPU"):
        fp4.cross_entropy_gemm(x, x, t)
    with pytest.raises(TypeError, match="dtype"):
        fp4.cross_entropy_gemm(x.float(), x, t)
    with pytest.raises(ValueError, match="on a GPU"):
        fp4.adapter_gemm(x, x, x, x, t)
    with pytest.raises(TypeError):
        fp4.rms_norm_backward_workspace_size(4, 4, torch.float16)


def test_binding_takes_every_argument_by_position():
    native = fp4.lm._binding()
    for name, count in (("rms_norm", 6), ("rms_norm_quantize", 7), ("rms_norm_backward", 7), ("cross_entropy_gemm", 6),
                        ("cross_entropy_gemm_backward", 9), ("adapter_gemm", 8)):
        f = getattr(native, name)
        with pytest.raises(TypeError, match="expected"):
            f(*[None] * (count - 1))
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            f(*[None] * count)
