"""The sizes of loss_plans.py reach the kernels that they are listed for (no GPU needed)."""
import pytest
import torch

from tests import loss_plans as plans
from tests.ffn_plans import TILES


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256,
                    reason="the plans are for 256 compute units")
def test_sizes_reach_their_kernels():
    for size, *want in plans.SIZES:
        assert list(plans.products(*size)) == want, size


def test_every_tile_is_reached():
    forward, prob = (set(p[i] for p in plans.SIZES) for i in (1, 2))
    assert forward == {"256", "128", "64x128", "64x128Long"}
    assert prob == set(TILES)
    many, few = ([p for p in plans.SIZES if (p[0][0] > 128) == b] for b in (True, False))
    assert {p[3] for p in many} == {(t, s) for t in TILES for s in (False, True)} | {plans.BOTH, plans.BOTH_SPLIT}
    assert {p[4] for p in many} == set(TILES) | {plans.BOTH, plans.BOTH_SPLIT}
    # of few rows' tiles those that any size was found for
    small = {"64", "64Deep", "64Long", "64x128", "64x128Long"}
    assert {p[3] for p in few} >= {(t, s) for t in small for s in (False, True)} | {plans.BOTH, plans.BOTH_SPLIT}
    assert {p[4] for p in few} >= {"64", "64x128", "128", "256", plans.BOTH, plans.BOTH_SPLIT}
