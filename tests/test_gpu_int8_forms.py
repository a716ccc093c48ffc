"""Forms of the 8-bit products and of the rows' quantization that few sizes
reach: every wide tile by expert, found by scans and by a plan, and rows of codes
that four waves make.  References and bounds are those of test_gpu_int8.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402
from int8_picks import FORMS  # noqa: E402
from test_gpu_int8 import TD, Problem, quantize_and_check  # noqa: E402


@pytest.mark.parametrize("case,want", FORMS, ids=lambda v: str(v)[:28])
def test_forms(case, want):
    rows, K, N, groups = case
    for act, k, dtype in (("none", 0, "bf16"), ("swiglu", 3, "f32")):
        p = Problem(rows, K, N, dtype, act=act, groups=groups, gather_k=k, bias=True, gap=1, seed=k)
        first = p.run()[:rows - 5].clone()
        p.check()
        assert torch.equal(p.run()[:rows - 5], first)


# (four waves to a row: more than 256 rows of more than 256 pieces of 16 bytes; from 4096 fp32 or 8192 bf16 columns
# on the rows do not stay in registers whole)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(257, 2051), (300, 7168), (513, 8200), (260, 20001), (301, 1025), (258, 4096)])
def test_quantize_wide_rows(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    ld = (cols + 7) // 8 * 8 + 8
    x = torch.full((rows, ld), float("nan"), dtype=TD[dtype])
    x[:, :cols] = torch.empty(rows, cols).normal_(generator=g).to(TD[dtype])
    x[:, :cols] *= torch.exp2(torch.randint(-60, 60, (rows, 1), generator=g).float()).to(TD[dtype])
    at = torch.randint(0, cols, (rows,), generator=g)
    x[torch.arange(rows), at] *= 64            # (the largest value in every wave's share)
    x[3, :cols] = 0
    x[4, cols - 1] = float("inf")
    x[5, 0] = float("nan")
    x[6, cols // 2] = float("-inf")
    x[rows - 1, :cols] = 0
    x[rows - 1, cols - 1] = -3
    quantize_and_check(x.to(DEV), cols, 1)
