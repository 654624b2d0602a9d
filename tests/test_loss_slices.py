"""The K slices of dX's product that the GPU runs are those that were planned (no GPU needed).

The number of slices is chosen on the host for all M rows and, where fewer take part, formed anew on the GPU (splits_of in
csrc/dense_tile.hpp).  The plan's tile is the best one only with the plan's slices, and its partial sums and their
reduction are paid for with any number of them.
"""
import ctypes
import random

import pytest
import torch

from tests import loss_plans as plans
from tests.ffn_plans import TILES, Plan, internal

pytestmark = pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256,
                                reason="the plans are for 256 compute units")
MOST = 16


class InputPlan(ctypes.Structure):
    _fields_ = [("plan", Plan), ("most", ctypes.c_int)]


def input_plan(m, k, cols):
    return internal("_ZN4fp4g15loss_input_planElll", InputPlan, 3)(m, k, cols)


def tile_rows(tile):
    return plans.ROWS.get(TILES[tile], 64)


def slices(p, m, rows):
    """splits_of for `rows` of m rows."""
    bm = tile_rows(p.plan.tile)
    return min(p.most, p.plan.S * -(-m // bm) // max(1, -(-rows // bm)))


def sizes():
    r = random.Random(1)
    return [s for s, *_ in plans.SIZES] + [(int(2 ** r.uniform(0, 13)), int(2 ** r.uniform(0, 15)), 8 * int(2 ** r.uniform(0, 10)))
                                           for _ in range(2000)]


def test_all_rows_have_the_planned_slices():
    split = 0
    for m, v, k in sizes():
        p = input_plan(m, k, v)
        assert slices(p, m, m) == p.plan.S and p.plan.S <= p.most <= MOST, (m, v, k, p.plan.S, p.most)
        split += p.plan.S > 1
    assert split > 50


def test_fewer_rows_have_as_many_or_more_within_the_workspace():
    for m, v, k in sizes()[::7]:
        p = input_plan(m, k, v)
        if p.plan.S == 1:
            continue
        for rows in {0, 1, m // 7, m // 2, m}:
            n = slices(p, m, rows)
            assert p.plan.S <= n <= MOST and n * rows <= p.plan.S * -(-m // 256) * 256, (m, v, k, rows, n)


def test_the_listed_sizes_run_as_they_are_listed():
    """One launch for both gradients among them: a split dX has more than one slice there."""
    for (m, v, k), _, _, x, _ in plans.SIZES:
        p = input_plan(m, k, v)
        assert (slices(p, m, m) > 1) == x[1], (m, v, k)
        assert x[0] in ("both", TILES[p.plan.tile]), (m, v, k)
