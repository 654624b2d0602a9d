"""Every kernel of the feed-forward products is reached by a size that the GPU tests run (tests/ffn_plans.py)."""
import pytest
import torch

from tests import ffn_plans as plans

ALL = {(tile, split) for tile in plans.TILES for split in (False, True)}


def reached(chosen):
    return {(tile, slices > 1) for tile, slices in chosen}


# The plan depends on the number of compute units; without a GPU the library assumes 256.
pytestmark = pytest.mark.skipif(
    torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256,
    reason="the listed sizes are those of 256 compute units")


@pytest.mark.parametrize("cases,elem,gates", [(plans.W8A8, 1, 1), (plans.W8A8_GATED, 1, 2), (plans.GATED, 2, 2)])
def test_products(cases, elem, gates):
    for size, tile, slices in cases:
        assert plans.product(*size, elem, gates) == (tile, slices), size
    assert reached((tile, slices) for _, tile, slices in cases) == ALL


def test_gradients():
    for size, x, w, merged in plans.GRADIENTS:
        assert plans.gradients(*size) == (x, w, merged), size
    assert reached(x for _, x, _, merged in plans.GRADIENTS if not merged) == ALL
    assert reached(w for _, _, w, merged in plans.GRADIENTS if not merged) == ALL
    assert reached(x for _, x, _, merged in plans.GRADIENTS if merged) == {
        (tile, split) for tile in ("64", "64Deep", "64x128") for split in (False, True)}
