"""The library's choice among its product kernels, and sizes that reach every one of them.

``dense_plan``, ``grad_plan``, ``gemv_takes`` and ``gemv_splits`` are the library's own host functions
(csrc/ffn_internal.h), so a change of their model cannot leave a listed size on another kernel unnoticed.
"""
import ctypes

import block_scaled_precision_e2m1_amd as fp4

TILES = ("256", "128", "128Deep", "64x128", "64Deep", "64", "64x128Long", "64Long")


class Plan(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int), ("S", ctypes.c_int), ("us", ctypes.c_double)]


class Grad(ctypes.Structure):
    _fields_ = [("x", Plan), ("w", Plan), ("merged", ctypes.c_bool)]


def internal(symbol, result, count):
    f = getattr(fp4.load_library(), symbol)
    f.restype, f.argtypes = result, [ctypes.c_int64] * count
    return f


def product(m, n, k, elem, gates, cap=16):
    """(tile, slices) of a product of operands of `elem` bytes with `gates` weights."""
    if internal("_ZN4fp4g10gemv_takesEllll", ctypes.c_bool, 4)(m, n, k * elem, gates):
        return "gemv", internal("_ZN4fp4g11gemv_splitsElllll", ctypes.c_int, 5)(m, n, k * elem, gates, cap)
    p = internal("_ZN4fp4g10dense_planElllll", Plan, 5)(m, gates * n, 1, -(-k * elem // 128), cap)
    return TILES[p.tile], p.S


def gradients(m, n, k, cap=16):
    """((tile, slices) of dX, (tile, slices) of dWg and dWu, both in one launch)."""
    p = internal("_ZN4fp4g9grad_planElllll", Grad, 5)(m, n, k, cap, cap)
    return (TILES[p.x.tile], p.x.S), (TILES[p.w.tile], p.w.S), p.merged


# Sizes with more than one tile and a ragged end in every dimension, one for each tile without and with a K split;
# slices of unequal length.
W8A8 = [((16493, 129, 16), "128", 1), ((199, 8413, 6704), "128", 3), ((12363, 209, 912), "128Deep", 1),
        ((2709, 129, 11456), "128Deep", 4), ((397, 25227, 144), "256", 1), ((391, 9369, 5536), "256", 3),
        ((65, 65, 16), "64", 1), ((65, 69, 2080), "64", 4), ((65, 65, 1072), "64Deep", 1), ((65, 65, 16848), "64Deep", 16),
        ((273, 357, 2208), "64Long", 1), ((547, 65, 26560), "64Long", 12), ((65, 8203, 288), "64x128", 1),
        ((65, 1379, 4672), "64x128", 8), ((65, 8315, 2784), "64x128Long", 1), ((65, 2723, 10544), "64x128Long", 4)]
W8A8_GATED = [((16721, 65, 16), "128", 1), ((8559, 97, 7072), "128", 3), ((259, 4981, 912), "128Deep", 1),
              ((2715, 67, 10544), "128Deep", 4), ((387, 12881, 144), "256", 1), ((9835, 193, 5136), "256", 3),
              ((65, 33, 16), "64", 1), ((67, 33, 2064), "64", 4), ((65, 35, 1040), "64Deep", 1),
              ((65, 33, 16448), "64Deep", 16), ((1087, 45, 2192), "64Long", 1), ((65, 267, 26528), "64Long", 12),
              ((65, 4185, 272), "64x128", 1), ((67, 325, 9280), "64x128", 16), ((65, 4237, 2576), "64x128Long", 1),
              ((65, 1357, 10352), "64x128Long", 4)]
GATED = [((131, 8333, 8), "128", 1), ((193, 4217, 3336), "128", 3), ((259, 4939, 456), "128Deep", 1),
         ((2805, 65, 5264), "128Deep", 4), ((389, 12549, 72), "256", 1), ((8207, 229, 2576), "256", 3),
         ((65, 33, 8), "64", 1), ((71, 33, 1056), "64", 4), ((65, 35, 536), "64Deep", 1), ((67, 33, 8624), "64Deep", 16),
         ((805, 61, 1096), "64Long", 1), ((65, 275, 13136), "64Long", 12), ((67, 4263, 136), "64x128", 1),
         ((67, 337, 4616), "64x128", 16), ((65, 4415, 1304), "64x128Long", 1), ((65, 675, 10592), "64x128Long", 8)]
# The backward products: dX's tile and slices, dW's, one launch.  A split dX has slices across the end of dG.
GRADIENTS = [((4121, 199, 5256), ("128", 1), ("128", 3), False), ((451, 829, 2000), ("64Long", 1), ("128Deep", 1), False),
             ((5419, 1397, 136), ("64Long", 1), ("128Deep", 4), False), ((65, 12771, 400), ("64Long", 16), ("256", 1), False),
             ((2999, 399, 5360), ("256", 1), ("256", 3), False), ((3, 7685, 72), ("64Deep", 16), ("64", 1), False),
             ((2261, 65, 72), ("64", 1), ("64", 8), False), ((1025, 93, 3720), ("64x128", 1), ("64Deep", 1), False),
             ((8375, 65, 72), ("64x128", 1), ("64Deep", 16), False), ((1371, 65, 1160), ("64x128", 1), ("64Long", 1), False),
             ((18543, 65, 72), ("64", 1), ("64Long", 16), False), ((201, 533, 3560), ("64Long", 1), ("64x128", 1), False),
             ((4793, 65, 328), ("64x128", 1), ("64x128", 16), False),
             ((1679, 67, 4104), ("128", 1), ("64x128Long", 1), False),
             ((10255, 65, 672), ("128", 1), ("64x128Long", 8), False), ((3, 8711, 136), ("64Long", 16), ("128", 1), False),
             ((8209, 1743, 200), ("128", 3), ("128Deep", 4), False), ((9973, 193, 264), ("128Deep", 1), ("64Long", 6), False),
             ((193, 9573, 648), ("128Deep", 16), ("256", 1), False), ((385, 1371, 10632), ("256", 3), ("256", 1), False),
             ((3077, 455, 8), ("64", 4), ("64", 12), False), ((2853, 261, 72), ("64Deep", 1), ("64", 8), False),
             ((65, 3869, 904), ("64x128", 16), ("128", 1), False),
             ((5495, 647, 136), ("64x128Long", 1), ("64Long", 3), False),
             ((65, 2719, 2728), ("64x128Long", 4), ("256", 1), False),
             ((65, 65, 72), ("64", 1), ("64", 1), True), ((67, 519, 72), ("64", 4), ("64", 1), True),
             ((65, 261, 72), ("64Deep", 1), ("64Deep", 1), True), ((519, 643, 72), ("64Deep", 4), ("64Deep", 1), True),
             ((65, 65, 2848), ("64x128", 1), ("64x128", 1), True), ((65, 2089, 136), ("64x128", 16), ("64x128", 1), True)]
