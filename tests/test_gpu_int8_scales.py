"""Products in 8-bit integers whose scales lie near fp32's ends: z has to be right
wherever fp32 holds it, whatever the sum times one of the two scales would be.
References and bounds are those of test_gpu_int8.py (scaling by powers of 2 is
exact, so no rounding is added to them)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402
from test_gpu_int8 import Problem  # noqa: E402


SCALED = [dict(rows=3, K=700, N=301), dict(rows=8, K=1031, N=130, act="swiglu"), dict(rows=5, K=300, N=67, groups=[2, 0, 3]),
          dict(rows=300, K=1000, N=513), dict(rows=700, K=640, N=2050, act="swiglu"),
          dict(rows=53, K=2762, N=4826), dict(rows=2045, K=2050, N=7170), dict(rows=200, K=5625, N=1402, act="swiglu",
                                                                               groups=[100, 0, 3, 1, 0, 16, 80, 0])]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", [-120, -100, 95, 97, 126])
@pytest.mark.parametrize("kw", SCALED, ids=lambda kw: f"{kw['rows']}x{kw['K']}x{kw['N']}")
def test_scales_far_apart(kw, power, dtype):
    """Rows of 2^power and weights of 2^-power: z stays near 1 while the sum times one scale alone would leave fp32."""
    p = Problem(**kw, dtype=dtype, bias=True, seed=power & 31)
    p.xs *= 2.0 ** power
    p.xs[::2] *= -1.0
    p.ws *= 2.0 ** -power
    p.x[1] = 0                                 # sums of 0: no infinity may stand on the way to them
    assert p.xs.isfinite().all() and p.ws.isfinite().all() and (p.ws != 0).all()
    p.run()
    p.check()


def test_large_rows_from_their_codes():
    """Rows near bf16's largest values, quantized, through weights small enough for the result."""
    g = torch.Generator().manual_seed(5)
    for rows in (2, 150):
        K, N = 512, 200
        x = (torch.empty(rows, K).uniform_(-1, 1, generator=g) * 3e38).bfloat16().to(DEV)
        c, s = torch.empty(rows, K, dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
        ds4.quantize_rows_int8(rows, K, x, c, s)
        w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).to(DEV)
        ws = torch.full((N,), 1e-35, device=DEV)
        y = torch.empty(rows, N, device=DEV)
        m = ds4.make_matmul_int8(K, N, dtype="f32")
        n = ds4.matmul_int8_workspace_bytes(m, rows)
        ds4.linear_int8(m, rows, c, s, w, ws, y, workspace=torch.empty(max(n, 16), dtype=torch.uint8, device=DEV))
        want = torch.matmul(c.double(), w.double().t()) * s.double()[:, None] * ws.double()
        assert ((y.double() - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all()


def test_infinite_and_nan_scales_stay_what_they_are():
    for rows in (4, 300):
        p = Problem(rows, 256, 96, "f32", seed=rows)
        p.xs[0], p.xs[1], p.xs[2] = float("inf"), float("nan"), float("-inf")
        p.x[3] = 0
        p.ws[0, 5] = float("inf")
        p.run()
        s = torch.matmul(p.x.double(), p.w[0].double().t())
        want = s * p.xs.double()[:, None] * p.ws.double()
        assert torch.equal(p.y.isnan(), want.isnan())
        assert torch.equal(p.y.isinf(), want.isinf()) and torch.equal(p.y[want.isinf()].double(), want[want.isinf()])
