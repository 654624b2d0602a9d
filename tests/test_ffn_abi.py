"""Host-side checks of the feed-forward entry points (include/fp4g_ffn.h): the library
exports what the header declares and refuses invalid arguments with the documented status
before touching a device (no GPU needed: nothing here passes validation with work to do)."""
import ctypes
import os
import re

import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp4g_ffn.h")

OK, EINVAL, EUNSUP, EALIGN = 0, 1, 2, 3
F32, BF16 = 0, 1
# Fake, aligned, non-overlapping "device" addresses: validation never dereferences them.
P = [0x10000000 * i for i in range(1, 16)]


@pytest.fixture(scope="module")
def lib():
    return fp4.ffn._library()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return set(re.findall(r"^\s*fp4g_status\s+([a-z_0-9]+)\s*\(", text, re.M))


def test_header_binding_and_library_agree(lib):
    assert declared() == set(fp4.FFN_SYMBOLS)
    for name in declared():
        assert hasattr(lib, name) and hasattr(fp4, name)


def quantize(lib, rows=4, K=64, X=P[0], t=BF16, c=P[1], s=P[2]):
    return lib.int8_quantize(rows, K, X, t, c, s, None)


def test_quantize_refusals(lib):
    assert quantize(lib, rows=-1) == EINVAL
    assert quantize(lib, K=-16) == EINVAL
    assert quantize(lib, rows=1 << 31) == EINVAL
    assert quantize(lib, rows=1 << 30, K=1 << 30) == EINVAL
    assert quantize(lib, K=24) == EUNSUP
    assert quantize(lib, t=2) == EINVAL
    assert quantize(lib, X=None) == EINVAL
    assert quantize(lib, c=None) == EINVAL
    assert quantize(lib, s=None) == EINVAL
    assert quantize(lib, X=P[0] + 8) == EALIGN
    assert quantize(lib, c=P[1] + 4) == EALIGN
    assert quantize(lib, s=P[2] + 2) == EALIGN
    assert quantize(lib, c=P[0] + 64) == EINVAL          # codes inside X
    assert quantize(lib, s=P[1] + 16) == EINVAL          # scales inside codes
    assert quantize(lib, rows=0, X=None, c=None, s=None) == OK


def gemm(lib, M=4, N=8, K=64, A=P[0], sa=P[1], B=P[2], sb=P[3], D=P[4], t=BF16, w=None, wb=0):
    return lib.w8a8_gemm(M, N, K, A, sa, B, sb, D, t, w, wb, None)


def gated8(lib, M=4, N=8, K=64, A=P[0], sa=P[1], Bg=P[2], sg=P[3], Bu=P[4], su=P[5], act=0, D=P[6], t=BF16, w=None, wb=0):
    return lib.w8a8_gated_gemm(M, N, K, A, sa, Bg, sg, Bu, su, act, D, t, w, wb, None)


@pytest.mark.parametrize("call", [gemm, gated8])
def test_int8_product_refusals(lib, call):
    assert call(lib, M=-1) == EINVAL
    assert call(lib, N=1 << 31) == EINVAL
    assert call(lib, M=1 << 30, N=1 << 30) == EINVAL
    assert call(lib, K=40) == EUNSUP
    assert call(lib, K=1 << 17) == EUNSUP                # 32-bit sums could overflow
    assert call(lib, t=2) == EINVAL
    assert call(lib, A=None) == EINVAL
    assert call(lib, sa=None) == EINVAL
    assert call(lib, D=None) == EINVAL
    assert call(lib, A=P[0] + 8) == EALIGN
    assert call(lib, sa=P[1] + 1) == EALIGN
    assert call(lib, D=P[8] + 2) == EALIGN
    assert call(lib, D=P[0]) == EINVAL
    assert call(lib, D=P[1]) == EINVAL
    assert call(lib, w=P[0], wb=1024) == EINVAL          # workspace over an input
    assert call(lib, w=P[9] + 4, wb=1024) == EALIGN
    assert call(lib, w=None, wb=1024) == EINVAL
    assert call(lib, M=0, A=None, sa=None, D=None) == OK
    assert call(lib, N=0, D=None) == OK


def test_gated_weights_and_activation_refusals(lib):
    assert gated8(lib, act=3) == EINVAL
    assert gated8(lib, act=-1) == EINVAL
    for name in ("Bg", "sg", "Bu", "su"):
        assert gated8(lib, **{name: None}) == EINVAL
    assert gated8(lib, Bu=P[4] + 1) == EALIGN
    assert gated8(lib, su=P[5] + 2) == EALIGN
    assert gated8(lib, D=P[4]) == EINVAL


def gated(lib, M=4, N=8, K=64, X=P[0], Wg=P[1], Wu=P[2], act=0, H=P[3], G=None, U=None, w=None, wb=0):
    return lib.gated_gemm(M, N, K, X, Wg, Wu, act, H, G, U, w, wb, None)


def test_gated_gemm_refusals(lib):
    assert gated(lib, K=-8) == EINVAL
    assert gated(lib, K=12) == EUNSUP
    assert gated(lib, K=1 << 22) == EUNSUP               # rows past 2^22 bytes
    assert gated(lib, act=7) == EINVAL
    assert gated(lib, G=P[4]) == EINVAL                  # one of G and U alone
    assert gated(lib, U=P[4]) == EINVAL
    for name in ("X", "Wg", "Wu", "H"):
        assert gated(lib, **{name: None}) == EINVAL
    for name, base in (("X", P[0]), ("Wg", P[1]), ("Wu", P[2]), ("H", P[3])):
        assert gated(lib, **{name: base + 2}) == EALIGN
    assert gated(lib, G=P[4] + 4, U=P[5]) == EALIGN
    assert gated(lib, H=P[1]) == EINVAL
    assert gated(lib, G=P[4], U=P[4] + 16) == EINVAL     # outputs over each other
    assert gated(lib, M=0, X=None, H=None) == OK


def backward(lib, M=4, N=8, K=64, dH=P[0], X=P[1], Wg=P[2], Wu=P[3], G=P[4], U=P[5], act=0, dX=P[6], dWg=P[7], dWu=P[8],
             w=P[9], wb=1 << 20):
    return lib.gated_gemm_backward(M, N, K, dH, X, Wg, Wu, G, U, act, dX, dWg, dWu, w, wb, None)


def test_backward_refusals(lib):
    assert backward(lib, M=-1) == EINVAL
    assert backward(lib, K=20) == EUNSUP
    assert backward(lib, N=(1 << 21) + 1) == EUNSUP      # rows of dG past 2^22 bytes
    assert backward(lib, act=3) == EINVAL
    for name in ("dH", "X", "Wg", "Wu", "G", "U", "dX", "dWg", "dWu", "w"):
        assert backward(lib, **{name: None}) == EINVAL
    assert backward(lib, dX=P[6] + 8) == EALIGN
    assert backward(lib, dX=P[1]) == EINVAL
    assert backward(lib, dWg=P[8]) == EINVAL
    assert backward(lib, w=P[6]) == EINVAL
    assert backward(lib, wb=4 * 4 * 64 - 1) == EINVAL    # less than dG and dU take
    assert backward(lib, K=0) == OK


def test_workspace_queries_validate(lib):
    n, m = ctypes.c_size_t(7), ctypes.c_size_t(7)
    for name in ("w8a8_gemm_workspace_size", "w8a8_gated_gemm_workspace_size", "gated_gemm_workspace_size"):
        f = getattr(lib, name)
        assert f(-1, 4, 64, ctypes.byref(n)) == EINVAL
        assert f(4, 4, 20, ctypes.byref(n)) == EUNSUP
        assert f(4, 4, 64, None) == EINVAL
        assert f(0, 4, 64, ctypes.byref(n)) == OK and n.value == 0
    f = lib.gated_gemm_backward_workspace_size
    assert f(4, 4, 64, ctypes.byref(n), None) == EINVAL
    assert f(0, 4, 64, ctypes.byref(n), ctypes.byref(m)) == OK and n.value == 0 and m.value == 0


def test_python_checks_come_before_the_library():
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fp4.int8_quantize(cpu)                           # not on a GPU
    with pytest.raises(TypeError):
        fp4.int8_quantize(None)
    with pytest.raises(TypeError):
        fp4.gated_gemm(cpu.half(), cpu, cpu) if torch.cuda.is_available() else fp4.gated_gemm(3, cpu, cpu)


def test_binding_takes_every_argument_by_position():
    """The compiled functions behind ffn.py: their names, and counts that are refused."""
    native = fp4.ffn._binding()
    for name, count in (("int8_quantize", 3), ("w8a8_gemm", 7), ("w8a8_gated_gemm", 10), ("gated_gemm", 7),
                        ("gated_gemm_backward", 8)):
        f = getattr(native, name)
        with pytest.raises(TypeError, match="expected"):
            f(*[None] * (count - 1))
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            f(*[None] * count)
