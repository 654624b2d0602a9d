"""The library's choice among its tiles for the loss's products, and sizes that reach every one of them.

The plans are the library's own host functions (csrc/ffn_internal.h, cross_entropy.hip), so a change of their model
cannot leave a listed size on another kernel unnoticed.
"""
import ctypes

import block_scaled_precision_e2m1_amd as fp4
from tests.ffn_plans import TILES, Plan, internal

ONE_GROUP = 1 << 0 | 1 << 1 | 1 << 3 | 1 << 6      # 256, 128, 64x128, 64x128Long: a wave has whole sums
ROWS = {"256": 256, "128": 128, "128Deep": 128}
BOTH, BOTH_SPLIT = ("both", False), ("both", True)


def products(m, v, k):
    """(forward tile, probabilities' tile, (dX's tile, whether K is split), dW's tile) for all of a vocabulary at once; both
    gradients of a small one go in one launch."""
    among = fp4.load_library()._ZN4fp4g16dense_plan_amongEjlllll
    among.restype, among.argtypes = Plan, [ctypes.c_uint32] + [ctypes.c_int64] * 5
    plan = internal("_ZN4fp4g10dense_planElllll", Plan, 5)
    forward, prob = among(ONE_GROUP, m, v, 1, -(-k // 64), 1), plan(m, v, 1, -(-k // 64), 1)
    terms = 2 if m <= 128 else 1                   # few rows: P in two terms along the contraction
    x, w = plan(m, k, 1, terms * -(-v // 64), 16), plan(v, k, 1, terms * -(-m // 64), 1)
    fx, fw = TILES[x.tile], TILES[w.tile]
    items = (-(-m // 64) * x.S + -(-v // 64)) * -(-k // 64)
    if ROWS.get(fx, 64) == 64 and ROWS.get(fw, 64) == 64 and items + 8 <= 512:
        return TILES[forward.tile], TILES[prob.tile], ("both", x.S > 1), ("both", x.S > 1)
    return TILES[forward.tile], TILES[prob.tile], (fx, x.S > 1), fw


# More than one 64 x 64 tile and a ragged end in every dimension.
SIZES = [
    ((71, 68, 8240), '64x128Long', '64Long', ('64x128', False), '64x128'),
    ((67, 2023, 456), '64x128', '64', ('64', True), '64'),
    ((664, 4894, 72), '128', '128', ('64x128', True), '64Deep'),
    ((386, 26319, 72), '256', '256', ('64Long', True), '64x128'),
    ((67, 10655, 688), '64x128', '64x128', ('64x128Long', True), '128'),
    ((8345, 67, 1352), '64x128Long', '64x128Long', ('128', False), '64Long'),
    ((70, 25038, 488), '64x128', '128Deep', ('64Long', True), '256'),
    ((67, 66, 528), '64x128', '64Deep', BOTH, BOTH),
    ((129, 66, 6984), '64x128Long', '64Long', ('64', False), '64'),
    ((1348, 16007, 72), '128', '128', ('128Deep', True), '64x128Long'),
    ((196, 3372, 8352), '64x128Long', '64Long', ('128', True), '256'),
    ((1602, 2759, 2536), '64x128', '64x128', ('256', True), '128'),
    ((136, 67, 72), '64x128', '64', BOTH, BOTH),
    ((68, 472, 72), '64x128', '64', BOTH_SPLIT, BOTH_SPLIT),
    ((141, 1002, 72), '64x128', '64', BOTH_SPLIT, BOTH_SPLIT),
    ((71, 70, 8080), '64x128Long', '64Long', ('64', False), '64'),
    ((67, 4360, 280), '64x128', '64', ('64Deep', True), '64x128'),
    ((69, 258, 4880), '64x128Long', '64Long', ('64Deep', False), '64x128'),
    ((142, 130, 5536), '64x128Long', '64Long', ('64x128', False), '64x128'),
    ((67, 596, 2720), '64x128Long', '64Long', ('64Long', False), '64x128'),
    ((70, 2414, 648), '64x128', '64Deep', ('64x128', True), '64x128'),
    ((138, 13229, 72), '128', '64', ('64Deep', True), '64x128'),
    ((132, 2062, 520), '64x128', '64Deep', ('64', True), '64x128'),
    ((132, 521, 2776), '64x128Long', '64Long', ('64Deep', False), '64x128'),
    ((129, 1175, 1464), '64x128Long', '64Long', ('64Long', False), '64x128'),
    ((71, 651, 8368), '64x128Long', '64Long', ('64x128Long', False), '128'),
    ((6588, 66, 1824), '64x128Long', '64Long', ('256', False), '64Long'),
    ((70, 8099, 1440), '64x128Long', '64Long', ('128Deep', True), '128'),
    ((472, 25055, 72), '256', '256', ('64Long', True), '128Deep'),
    ((131, 1286, 6048), '64x128Long', '64Long', ('64x128Long', False), '64x128'),
    ((2747, 5167, 72), '256', '256', ('64x128Long', True), '64Long'),
    ((1944, 450, 1552), '64x128Long', '64Long', ('128Deep', False), '64Long'),
]
