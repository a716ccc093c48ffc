"""Which kernel the library takes for a product in 8-bit integers, asked of the
built library itself (host code: no GPU is needed)."""
import ctypes

import bit_routed_moe_amd as ds4


class _Pick(ctypes.Structure):
    _fields_ = [("shape", ctypes.c_int), ("splits", ctypes.c_int), ("us", ctypes.c_double)]


def pick(rows, K, N, groups=1):
    """(shape, splits, plan): shape 0 .. 4 of the tiles 256x256, 128x256 (pipelined), 128x256, 128x128, 64x64, or -1
    for the few-row kernel; the parts of the contraction; whether a grouped call's chunks are listed by a launch of
    their own (else each workgroup scans for its chunk)."""
    lib = ctypes.CDLL(ds4.LIB_PATH)
    choose, plan = lib._ZN3ds47m8_pickEiiii, lib._ZN3ds413m8_wants_planERKNS_6M8PickEiii
    choose.restype, choose.argtypes = _Pick, [ctypes.c_int] * 4
    plan.restype, plan.argtypes = ctypes.c_bool, [ctypes.POINTER(_Pick)] + [ctypes.c_int] * 3
    p = choose(rows, K, N, groups)
    listed = p.shape >= 0 and groups > 1 and plan(ctypes.byref(p), rows, N, groups)
    return p.shape, p.splits, listed


# rows, K, N, rows of each group (5 rows more than they sum to), and what the product takes.  Of each wide tile a
# group of whole chunks, ends of every kind (1 row, one short of 16, one more than the tile) and groups without rows;
# contractions that end inside a stage and that fill it; the most groups, listed by a plan launch.
FORMS = [
    ((360, 3127, 1254, [200, 128, 1, 15, 0, 11] + [0] * 63), (2, 1, False)),
    ((360, 3136, 1254, [0] * 60 + [128, 113, 112, 0, 2, 0, 0, 0, 0]), (2, 1, False)),
    ((7151, 7036, 4240, [3000, 0, 129, 128, 1, 2500, 1200, 95, 93]), (2, 1, True)),
    ((7151, 7040, 4242, [0, 256, 255, 257, 4096, 0, 1000, 1282, 0]), (2, 1, True)),
    ((5615, 1547, 2728, [5610, 0]), (0, 1, False)),
    ((16245, 1626, 4812, [257, 15983]), (0, 1, True)),
    ((3769, 3611, 1922, [129, 3635]), (1, 1, False)),
    ((6520, 4451, 5718, [1, 6514]), (1, 1, True)),
    ((28623, 145, 130, [0, 1, 63, 64, 65, 3] * 3 + [20000, 0] + [0, 16] * 498 + [58, 0, 0, 0, 0, 0, 0, 4]), (4, 1, True)),
    ((36417, 71, 134, [0, 1, 127, 128, 129, 3] * 3 + [20000, 0] + [0, 30] * 498 + [301, 0, 0, 0, 0, 0, 1, 6]), (3, 1, True)),
]
