"""Products whose operands are +1 and -1, so that every sum is a small whole
number: fp32 sums of up to 2^24 of them are exact in any order, a result has to
equal the exact one (rounded once where it is bf16), and a term that is left
out or taken twice changes it.  Then the error's norm on random operands, which
sums in too few bits would raise."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402
from test_gpu_matmul import EVAL, HALF, TD, Problem, act64  # noqa: E402


def signs(t, g):
    if t is not None:
        t.copy_(torch.randint(0, 2, t.shape, generator=g) * 2 - 1)


class Signs(Problem):
    """A Problem of +1 and -1 (also z, so that relu passes half of dy on)."""

    def __init__(self, *args, seed=0, **kw):
        super().__init__(*args, seed=seed, **kw)
        assert self.act in ("none", "relu")
        g = torch.Generator().manual_seed(seed + 1)
        for t in (self.x, self.w, self.bias, self.res, self.dy, self.zin):
            signs(t, g)

    def same(self, name, got, want):
        wrong = (got.double() != want.to(got.dtype).double()).nonzero()
        assert len(wrong) == 0, (name, len(wrong), wrong[:3].tolist(), want.shape)

    def check_forward(self):
        x, w = self.x.double()[self.src.to(DEV)], self.w.double()
        for e in range(self.E):
            a, b = self.off_h[e], self.off_h[e + 1]
            z = x[a:b] @ w[e].t()
            z = z if self.bias is None else z + self.bias[e].double()
            y = z if self.act == "none" else z.clamp(min=0)
            y = y if self.res is None else y + self.res[a:b].double()
            if self.save:
                self.same("z", self.z[a:b], z)
            self.same("y", self.y[a:b], y)
        self._outside(self.y)

    def check_backward(self, dx=True, dw=True, dbias=True):
        x, w = self.x.double()[self.src.to(DEV)], self.w.double()
        for e in range(self.E):
            a, b = self.off_h[e], self.off_h[e + 1]
            dz = self.dy[a:b].double()
            dz = dz if self.act == "none" else dz * (self.zin[a:b].double() > 0)
            if dx:
                self.same("dx", self.dx[a:b], dz @ w[e])
            if dw:
                self.same("dw", self.dw[e], dz.t() @ x[a:b])
            if dbias:
                self.same("dbias", self.dbias[e], dz.sum(0))
        if dx:
            self._outside(self.dx)


def run_both(p, backward=True):
    p.forward()
    p.check_forward()
    if backward:
        p.backward()
        p.check_backward()


# ends inside a tile, a stage, a 16-byte piece; splits of the contraction in each direction; every tile shape
@pytest.mark.parametrize("dtype,grad", [("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,K,N", [
    (1, 1, 1), (1, 1031, 333), (7, 130, 65), (16, 520, 259), (65, 65, 66), (100, 8192, 130), (129, 1000, 514),
    (40, 4104, 72), (70, 96, 4104), (4100, 72, 40), (1000, 1500, 700), (2045, 2050, 1026)])
def test_linear(rows, K, N, dtype, grad):
    for act in ("none", "relu"):
        print(f"exact linear {rows}x{K}->{N} {act} {dtype}", flush=True)
        run_both(Signs(rows, K, N, dtype, act, bias=True, residual=rows % 2 == 1, grad=grad, seed=rows))


@pytest.mark.parametrize("rows,K,N", [(4090, 2042, 2306), (1021, 1026, 7170), (4100, 1026, 4100)])
def test_linear_large(rows, K, N):
    print(f"exact linear {rows}x{K}->{N}", flush=True)
    run_both(Signs(rows, K, N, "bf16", "none", bias=True, grad="f32", seed=rows))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("groups", [[1], [0, 3, 0], [5, 130, 0, 64, 1], [1] * 40, [300, 0, 515, 2], [2, 4990, 0, 7]],
                         ids=lambda g: "-".join(map(str, g))[:20])
def test_grouped(groups, dtype):
    for K, N, k in ((136, 264, 3), (77, 51, 2), (520, 72, 0)):
        print(f"exact grouped {groups[:6]} {K}->{N} {dtype}", flush=True)
        run_both(Signs(sum(groups) + 3, K, N, dtype, "none", groups=groups, gather_k=k, bias=True, grad="f32",
                       seed=len(groups)))


# Weight gradients of gathered rows.  With few outputs the rows are split over up to 16 workgroups, which start
# anywhere in the ring of row numbers and fill it again every 1024 rows from row 2048 of a share on; large outputs
# take the 256-wide tiles with the same ring.
@pytest.mark.parametrize("K,N,groups", [
    (128, 128, [8192, 8190]), (128, 128, [39000, 1500]), (128, 128, [61, 16300]), (200, 200, [3000, 5190]),
    (500, 300, [12000, 5, 9000, 3570]), (72, 136, [33003]), (136, 72, [0, 16000, 383]),
    (2100, 1030, [6100, 2900]), (2060, 2060, [5200, 800]), (520, 1030, [2100, 0, 4700, 2200, 1, 2999])],
    ids=lambda g: "-".join(map(str, g)) if isinstance(g, list) else str(g))
@pytest.mark.parametrize("gather_k", [0, 2])
def test_weight_gradient_of_many_rows(K, N, groups, gather_k):
    print(f"exact dw {groups} {K}->{N} gather {gather_k}", flush=True)
    p = Signs(sum(groups) + 1, K, N, "bf16", "none", groups=groups, gather_k=gather_k, grad="f32", save=False, seed=K)
    p.backward(dx=False)
    p.check_backward(dx=False)
    first = p.dw.clone()
    p.dw.fill_(float("nan"))
    p.backward(dx=False, dbias=False)
    assert torch.equal(first, p.dw)


# Norm of the error over the norm of the result, on random operands:
#   a rounding to b bits of independent values moves each by at most half a step, evenly spread over the step: its
#     norm is at most half a step / sqrt(3) of the result's, 5% more for the spread over some thousand results;
#   n additions in fp32 each move a partial sum, no larger than the result in the mean, by at most 2^-23 (a rounding,
#     or a cut) to either side: sqrt(n) * 2^-23;
#   an activation adds 16 * 2^-24 of its own, and may leave values a quarter of z's size: 4 times the sums' error;
#   dz, taken here from fp64 and rounded to bf16, may be rounded to the other side: an error e before a rounding to
#     steps of s does that with probability 2 e / s and leaves s, in the mean square 2 e s, with
#     e <= 2^-20 |dy| (1 + |z|)^2 and s <= 2^-7 |dz|; for z of deviation 1.5 the mean of (1 + |z|)^2 is 5.7 and
#     |dy| / |dz| is about 2 (in the mean square): sqrt(2 * 2^-20 * 2^-7 * 5.7 * 2) = 4.2e-4, below 2^-11;
#   e itself, where dz is not rounded, has 7.5 for the root of the mean of (1 + |z|)^4: 2^-20 * 7.5 * 2 < 2^-16.
def norm_limit(dtype, n, act, dz=0.0):
    lim = 1.05 / math.sqrt(3) * HALF[dtype] + math.sqrt(n) * 2.0 ** -23 * (1 if act == "none" else 4)
    return lim if act == "none" else lim + EVAL + dz


def norm_check(name, got, want, limit):
    err = ((got.double() - want).norm() / want.norm()).item()
    assert err <= limit, (name, err, limit)


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("act", ["none", "swiglu", "gelu_tanh"])
@pytest.mark.parametrize("rows,K,N,groups,gather_k", [
    (100, 8192, 130, None, 0), (4100, 72, 40, None, 0), (600, 520, 264, None, 0),
    (5003, 72, 40, [2, 4990, 0, 7], 2), (3000, 136, 96, [1500, 3, 1497], 3), (70, 96, 4104, None, 0)])
def test_error_norms(rows, K, N, groups, gather_k, act, dtype, grad):
    print(f"norms {rows}x{K}->{N} {act} {dtype} {grad}", flush=True)
    p = Problem(rows, K, N, dtype, act, groups=groups, gather_k=gather_k, bias=True, grad=grad, seed=rows + 1)
    p.forward()
    p.backward()
    x, w = p.x.double()[p.src.to(DEV)], p.w.double()
    end = p.off_h[-1]
    z, dz, dx, dw, db = [], [], [], [], []
    for e in range(p.E):
        a, b = p.off_h[e], p.off_h[e + 1]
        z.append(x[a:b] @ w[e].t() + p.bias[e].double())
        d = p.dy[a:b].double()
        if act != "none":
            v = p.zin[a:b].double().requires_grad_()
            d, = torch.autograd.grad(act64(v, act), v, d)
        db.append(d.sum(0))
        d = d.to(TD[dtype]).double() if dtype == "bf16" else d
        dx.append(d @ w[e])
        dw.append(d.t() @ x[a:b])
    z = torch.cat(z)
    norm_check("z", p.z[:end], z, norm_limit(dtype, K, "none"))
    norm_check("y", p.y[:end], act64(z, act), norm_limit(dtype, K, act))
    operand = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -16
    norm_check("dx", p.dx[:end], torch.cat(dx), norm_limit(dtype, N, act, operand))
    norm_check("dw", p.dw, torch.stack(dw), norm_limit(grad, rows, act, operand))
    norm_check("dbias", p.dbias, torch.stack(db), norm_limit(grad, rows, act, 2.0 ** -16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,N", [(3, 1 << 20, 24), (20, 1 << 20, 8), (2, 16, 1 << 20), (20, 8, (1 << 20) - 8)])
def test_largest_widths(rows, K, N, dtype):
    print(f"largest {rows}x{K}->{N} {dtype}", flush=True)
    run_both(Signs(rows, K, N, dtype, "none", bias=True, grad="f32", seed=7))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_most_rows(dtype):
    """2^24 rows, made on the GPU: every sum over them stays below 2^24."""
    rows, n = (1 << 24) - 5, 8
    print(f"most rows {dtype}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(5)
    mk = lambda *s: (torch.randint(0, 2, s, generator=g, device=DEV, dtype=torch.int8) * 2 - 1).to(TD[dtype])
    x, w, dy = mk(rows, n), mk(n, n), mk(rows, n)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    dw, db = torch.empty(n, n, device=DEV), torch.empty(n, device=DEV)
    m = ds4.make_matmul(n, n, dtype=dtype, grad="f32")
    ws = torch.empty(max(16, ds4.matmul_workspace_bytes(m, rows), ds4.matmul_workspace_bytes(m, rows, True)),
                     dtype=torch.uint8, device=DEV)
    ds4.linear(m, rows, x, w, y, workspace=ws)
    ds4.linear_backward(m, rows, x, w, dy, dx=dx, dw=dw, dbias=db, workspace=ws)
    assert torch.equal(y.float(), x.float() @ w.float().t()) and torch.equal(dx.float(), dy.float() @ w.float())
    assert torch.equal(dw.double(), dy.double().t() @ x.double()) and torch.equal(db.double(), dy.double().sum(0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [3, 200, 5000])
def test_1024_groups(rows, dtype):
    """The most groups, most of them empty or of a few rows."""
    g = torch.Generator().manual_seed(rows)
    groups = torch.bincount(torch.randint(0, 1024, (rows,), generator=g) // 3 * 3, minlength=1024).tolist()
    print(f"1024 groups, {rows} rows {dtype}", flush=True)
    run_both(Signs(rows + 2, 72, 40, dtype, "none", groups=groups, gather_k=2, bias=True, grad="f32", seed=rows))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [12, 700])
def test_nan_stays_in_its_rows_and_groups(rows, dtype):
    """NaN and infinities in rows of no group, in rows of x that no row reads and in one expert's operands reach no
    other result."""
    groups = [rows // 4, 0, rows // 2, rows - rows // 4 - rows // 2]
    p = Signs(rows + 3, 136, 72, dtype, "none", groups=groups, gather_k=2, bias=True, grad="f32", seed=rows)
    a, b, own = p.off_h[2], p.off_h[3], p.x_rows - 1
    src = p.src.clone()
    src[(src == 0) | (src == own)] = 1      # token 0 is read by no row, the last one by one of the third expert's
    src[a] = own
    p.src = src
    p.pairs.copy_((2 * src).to(torch.int32))
    p.x[0] = float("nan")
    p.dy[rows:] = float("inf")
    p.x[own] = float("nan")
    p.w[1] = float("inf")                   # an expert without rows
    p.dy[a] = float("nan")
    p.forward()
    p.backward()
    x, w = p.x.double()[p.src.to(DEV)], p.w.double()
    for e in (0, 3):
        i, j = p.off_h[e], p.off_h[e + 1]
        p.same("y", p.y[i:j], x[i:j] @ w[e].t() + p.bias[e].double())
        p.same("dx", p.dx[i:j], p.dy[i:j].double() @ w[e])
        p.same("dw", p.dw[e], p.dy[i:j].double().t() @ x[i:j])
        p.same("dbias", p.dbias[e], p.dy[i:j].double().sum(0))
    assert (p.dw[1] == 0).all() and (p.dbias[1] == 0).all()
    p.same("y", p.y[a + 1:b], x[a + 1:b] @ w[2].t() + p.bias[2].double())
    p.same("dx", p.dx[a + 1:b], p.dy[a + 1:b].double() @ w[2])
    for t in (p.y[a], p.dx[a], p.dw[2], p.dbias[2]):
        assert torch.isnan(t).all()
    assert torch.isnan(p.y[rows:]).all() and torch.isnan(p.dx[rows:]).all()   # (left as they were)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "swiglu"])
def test_extreme_preactivations(act, rows, dtype):
    """Activations and their derivatives where squares, exponentials and products leave fp32's range.  z is x itself
    (w the unit matrix), and dbias of one row is dz, unrounded.

    A value is off by 16 * 2^-24 of itself (EVAL), and where it falls as e^-t by 4 roundings of t, at most 88 before
    fp32's range ends; a derivative, whose terms cancel, by EVAL * (1 + |z|)^2, |z| counted up to 10 (behind that it
    is 0 or 1 to within e^-10 * 11).  Past t = 88.72 e^t leaves fp32's range and the value is 0, which is off by less
    than 88.73 * 2^-128 < 2^-121."""
    v = torch.tensor([0.0, 2e-38, 1e-4, 0.7, 2.0, 5.0, 9.5, 13.0, 20.0, 88.0, 90.0, 101.0, 1e4, 1e13, 1e20, 3e38])
    v = torch.cat([v, -v])
    n = len(v)
    if act == "swiglu":                      # each as the gate, and as the other factor
        q = torch.full((n,), 0.25)
        v = torch.cat([v, q, q, v])          # (gates: v and 1/4, then their partners)
    z = v.to(TD[dtype]).to(DEV)
    N = z.numel()
    oc = N // 2 if act == "swiglu" else N
    m = ds4.make_matmul(N, N, dtype=dtype, act=act, grad="f32")
    ws = torch.empty(max(16, ds4.matmul_workspace_bytes(m, rows), ds4.matmul_workspace_bytes(m, rows, True)),
                     dtype=torch.uint8, device=DEV)
    x = z.expand(rows, N).contiguous()
    y = torch.empty(rows, oc, dtype=TD[dtype], device=DEV)
    zs = torch.empty_like(x)
    ds4.linear(m, rows, x, torch.eye(N, dtype=TD[dtype], device=DEV), y, z=zs, workspace=ws)
    assert torch.equal(zs, x)
    zd = z.double()[None].requires_grad_()
    if act == "gelu_tanh":                   # 1 + tanh as 2 sigmoid: nothing cancels
        want = zd * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (zd + 0.044715 * zd ** 3))
    else:
        want = act64(zd, act)
    h = HALF[dtype]
    err = (y.double() - want).abs()
    bad = ~(err <= (EVAL + 88 * 2.0 ** -22 + h) * 1.01 * want.abs() + 2.0 ** -121)
    assert not bad.any(), (act, z[:oc][bad[0]].tolist(), y[0][bad[0]].tolist())
    dy = torch.full((1, oc), 0.5, dtype=TD[dtype], device=DEV)
    dbias = torch.empty(N, device=DEV)
    ds4.linear_backward(m, 1, None, None, dy, z=z[None].contiguous(), dbias=dbias, workspace=ws)
    dz, = torch.autograd.grad(want, zd, dy.double())
    a = zd.detach().abs().clamp(max=10)
    scale = (1 + a) ** 2
    if act == "swiglu":                      # the gate's derivative times u, and silu of the gate
        g, u = zd.detach().chunk(2, 1)
        scale = torch.cat([(1 + g.abs().clamp(max=10)) ** 2 * u.abs(), (g * torch.sigmoid(g)).abs()], 1)
    err = (dbias.double()[None] - dz).abs()
    bad = ~(err <= EVAL * 0.5 * scale + 2.0 ** -121)
    assert not bad.any(), (act, z[bad[0]].tolist(), dbias[bad[0]].tolist(), dz[bad].tolist())


def test_two_graphs_share_a_workspace():
    """A gathered product with its gradients (split contraction, refilled rings) and a dense one in two captured
    graphs over one workspace, replayed in turn with new inputs and eager calls between."""
    ps = [Signs(16390, 128, 128, "bf16", "relu", groups=[8192, 0, 8190], gather_k=2, bias=True, grad="f32", seed=3),
          Signs(100, 8192, 130, "bf16", "none", bias=True, grad="f32", seed=4)]
    n = max(ds4.matmul_workspace_bytes(p.m, p.rows, back) for p in ps for back in (False, True))
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV)

    def both(p):
        p.forward(ws=ws)
        p.backward(ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for p in ps:
            both(p)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both(p)
        graphs.append(g)
    gen = torch.Generator().manual_seed(9)
    for rep in range(6):
        for p, g in zip(ps, graphs):
            signs(p.x, gen)
            signs(p.dy, gen)
            for t in (p.y, p.z, p.dx, p.dw, p.dbias):
                t.fill_(float("nan"))
            ws.fill_(0x5A)
            torch.randn(1000, device=DEV).sum().item()
            g.replay()
            torch.cuda.synchronize()
            p.check_forward()
            p.check_backward()
