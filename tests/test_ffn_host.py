"""Host-side behaviour of the feed-forward operators beyond the refusals of test_ffn_abi.py (no GPU needed: every
call is refused before a launch)."""
import pytest

from tests.test_ffn_abi import EALIGN, EINVAL, P, backward, gated, gated8, gemm, lib  # noqa: F401


@pytest.mark.parametrize("call", [gemm, gated8, gated, backward])
@pytest.mark.parametrize("size", [1 << 63, (1 << 64) - 16, (1 << 64) - 1])
def test_workspace_sizes_past_63_bits(lib, call, size):  # noqa: F811
    """A size whose top bit is set is a size like any other: its buffer has to be there, aligned and clear of the inputs."""
    assert call(lib, w=None, wb=size) == EINVAL
    assert call(lib, w=P[10] + 4, wb=size) == EALIGN
    assert call(lib, w=P[0], wb=size) == EINVAL          # reaches over the inputs
    assert call(lib, w=P[0] - 16, wb=size) == EINVAL
