"""Which kernels the covering sizes of the 8-bit products' GPU tests take: a
change of the estimate that moves one of them to another kernel fails here, not
in silence there (no GPU)."""
import pytest

pytest.importorskip("bit_routed_moe_amd")
from int8_picks import FORMS, pick  # noqa: E402
from test_gpu_int8 import PARTS  # noqa: E402


@pytest.mark.parametrize("case,want", FORMS, ids=lambda v: str(v)[:28])
def test_forms(case, want):
    rows, K, N, groups = case
    assert sum(groups) + 5 == rows and len(groups) <= 1024
    assert pick(rows, K, N, len(groups)) == want


def test_parts():
    taken = set()
    for rows, K, N, groups in PARTS:
        taken.add(pick(rows, K, N) + ("dense",) if groups is None else pick(sum(groups) + 5, K, N, len(groups)) + ("groups",))
    assert taken >= {(0, 1, False, "dense"), (1, 1, False, "dense"), (3, 2, False, "dense"), (3, 4, False, "dense"),
                     (3, 8, False, "dense"), (4, 2, False, "dense"), (4, 4, False, "dense"), (4, 8, False, "dense"),
                     (4, 16, False, "dense"), (1, 1, False, "groups"), (2, 1, False, "groups"), (3, 4, True, "groups"),
                     (4, 2, True, "groups"), (4, 4, True, "groups"), (4, 8, True, "groups"), (4, 16, True, "groups")}


def test_few_rows_and_small_tiles():
    assert pick(1, 7168, 7168) == (-1, 1, False) and pick(16, 2048, 7168, 256) == (-1, 1, False)
    assert pick(130, 511, 130)[0] == -1 and pick(1000, 640, 2050) == (4, 1, False)
    assert pick(9000, 200, 64, 1024) == (4, 1, False)                    # (each workgroup scans 1024 groups)
