"""The most rows that the rows' quantization takes, wide enough for a workgroup
each: more than one dimension of a launch holds."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402
from test_gpu_int8 import reference_codes  # noqa: E402


def test_most_rows():
    rows, cols, ldx, ldq = 1 << 24, 2049, 2056, 2064
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("104 GB of tensors")
    x = torch.zeros(rows, ldx, dtype=torch.bfloat16, device=DEV)
    codes = torch.full((rows, ldq), 77, dtype=torch.int8, device=DEV)
    scale = torch.full((rows,), -5.0, device=DEV)
    at = torch.tensor([0, 1, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, rows - 2, rows - 1])
    some = torch.empty(len(at), cols).normal_(generator=torch.Generator().manual_seed(1)).bfloat16()
    for i, r in enumerate(at.tolist()):
        x[r, :cols] = some[i].to(DEV)
    ds4.quantize_rows_int8(rows, cols, x[:, :cols], codes[:, :cols], scale)
    q, s = reference_codes(some)
    for i, r in enumerate(at.tolist()):
        assert torch.equal(codes[r, :cols].cpu(), q[i]) and float(scale[r]) == float(s[i])
        codes[r, :cols] = 0
        scale[r] = 0
    assert not scale.any()                    # the rows of zeros: scale 0 and codes 0
    for part in codes.split(1 << 20):
        assert not part[:, :cols].any() and (part[:, cols:] == 77).all()
    del x, codes, scale, part
    torch.cuda.empty_cache()
