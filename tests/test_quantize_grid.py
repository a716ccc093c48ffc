"""The launches of the rows' quantization, asked of the built library's host
code (no GPU): every row is reached and no dimension has 2^32 threads, up to the
most rows that the call accepts; and the sizes of the GPU tests take each of the
kernel's forms."""
import ctypes

import pytest

ds4 = pytest.importorskip("bit_routed_moe_amd")


class Grid(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("waves", "threads", "x", "y")]


def grid(rows, cols, f32):
    f = ctypes.CDLL(ds4.LIB_PATH)._ZN3ds418quantize_rows_gridEiib
    f.restype, f.argtypes = Grid, [ctypes.c_int, ctypes.c_int, ctypes.c_bool]
    return f(rows, cols, f32)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("cols", [1, 1024, 1025, 2048, 2049, 7168, 1 << 20])
@pytest.mark.parametrize("rows", [1, 3, 256, 257, 1 << 20, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, (1 << 24) - 1, 1 << 24])
def test_every_row_within_the_limits(rows, cols, f32):
    g = grid(rows, cols, f32)
    at_once = g.threads // (64 * g.waves)
    assert at_once >= 1 and g.x * g.threads < 1 << 32 and 1 <= g.y <= 65535
    assert g.x * g.y * at_once >= rows and (g.x - 1) * g.y * at_once < rows


def test_forms_of_the_tests_sizes():
    for dtype in (False, True):
        assert grid(1000, 300, dtype).waves == 1 and grid(2, 40000, dtype).waves == 16
        for rows, cols in ((257, 2051), (300, 7168), (513, 8200), (260, 20001), (258, 4096)):
            assert grid(rows, cols, dtype).waves == 4
    assert grid(301, 1025, True).waves == 4
