"""Host-side behaviour of the feed-forward operators beyond the refusals of test_ffn_abi.py (no GPU needed: every
call is refused before a launch)."""
import ctypes
import shutil

import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4
from tests import ffn_plans as plans
from tests.test_ffn_abi import EALIGN, EINVAL, EUNSUP, OK, P, backward, gated, gated8, gemm, lib  # noqa: F401


@pytest.mark.parametrize("call", [gemm, gated8, gated, backward])
@pytest.mark.parametrize("size", [1 << 63, (1 << 64) - 16, (1 << 64) - 1])
def test_workspace_sizes_past_63_bits(lib, call, size):  # noqa: F811
    """A size whose top bit is set is a size like any other: its buffer has to be there, aligned and clear of the inputs."""
    assert call(lib, w=None, wb=size) == EINVAL
    assert call(lib, w=P[10] + 4, wb=size) == EALIGN
    assert call(lib, w=P[0], wb=size) == EINVAL          # reaches over the inputs
    assert call(lib, w=P[0] - 16, wb=size) == EINVAL


def test_launches_of_few_token_products_hold_their_threads():
    """Fewer than 2^32 threads a launch at the largest N, whatever K and M (256 threads a workgroup at most)."""
    takes = plans.internal("_ZN4fp4g10gemv_takesEllll", ctypes.c_bool, 4)
    splits = plans.internal("_ZN4fp4g11gemv_splitsElllll", ctypes.c_int, 5)
    for n in ((1 << 27) - 1, 1 << 26, 1 << 21, 1 << 20, 5000):
        for kb in (16, 1024, 65536, 1 << 22):
            for m in (1, 16, 32, 64):
                for gates in (1, 2):
                    if takes(m, n, kb, gates):
                        groups = -(-n // (32 if gates * n * kb >= 1 << 25 and n >= 32 * 171 else 16))
                        assert groups * splits(m, n, kb, gates, 16) * 256 < 1 << 32, (m, n, kb, gates)
    assert not takes(1, 1 << 27, 16, 1)


def test_backward_takes_two_million_channels_and_no_more(lib):  # noqa: F811
    n, least = ctypes.c_size_t(), ctypes.c_size_t()
    query = lib.gated_gemm_backward_workspace_size
    assert query(4, 1 << 21, 64, ctypes.byref(n), ctypes.byref(least)) == OK and least.value == 4 * 4 << 21
    assert query(4, (1 << 21) + 1, 64, ctypes.byref(n), ctypes.byref(least)) == EUNSUP
    assert backward(lib, N=(1 << 21) + 1, K=64) == EUNSUP
    assert lib.gated_gemm_workspace_size(4, (1 << 21) + 1, 64, ctypes.byref(n)) == OK


def test_a_wrong_type_is_a_type_error_wherever_the_tensor_is():
    """As for every other argument (the type, then the shape, then the device), and with or without a GPU."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: fp4.gated_gemm(x.half(), x, x), lambda: fp4.int8_quantize(x.half()),
                 lambda: fp4.w8a8_gemm(x, x, x, x), lambda: fp4.w8a8_gated_gemm(x, x, x, x, x, x),
                 lambda: fp4.gated_gemm_backward(x, x.float(), x, x, x, x)):
        with pytest.raises(TypeError, match="dtype"):
            call()
    with pytest.raises(ValueError, match="on a GPU"):
        fp4.gated_gemm(x, x, x)


def test_gradients_are_taken_at_any_element(lib):  # noqa: F811
    """dH, G and U are read at their elements' alignment; a workspace that is too small is found after it."""
    assert backward(lib, wb=16) == EINVAL
    for name, at, element in (("dH", P[0], 2), ("G", P[4], 4), ("U", P[5], 4)):
        assert backward(lib, **{name: at + element}, wb=16) == EINVAL
        assert backward(lib, **{name: at + element // 2}, wb=16) == EALIGN
    for name, at in (("X", P[1]), ("Wg", P[2]), ("Wu", P[3]), ("dX", P[6]), ("dWg", P[7]), ("dWu", P[8]), ("w", P[9])):
        assert backward(lib, **{name: at + 4}, wb=16) == EALIGN


def test_the_library_is_built_where_the_binding_cannot_be(monkeypatch):
    """No C++ compiler, or none of torch's headers: the library and the oracle are there, and the build says what is not."""
    import __graft_entry__ as entry
    import oracle
    from block_scaled_precision_e2m1_amd import _build
    done = []
    monkeypatch.setattr(_build, "build", lambda *a, **k: done.append("library"))
    monkeypatch.setattr(oracle, "build", lambda *a, **k: done.append("oracle"))
    monkeypatch.setattr(fp4, "load_library", lambda: done.append("loaded"))
    which = shutil.which
    monkeypatch.setattr(_build.shutil, "which", lambda name: None if name in ("g++", "c++") else which(name))
    with pytest.raises(RuntimeError, match="binding"):
        entry.build()
    assert done == ["library", "oracle", "loaded"]
