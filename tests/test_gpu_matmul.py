"""Products at original precision (ds4moe_linear, ds4moe_grouped_matmul and
their gradients) against the formulas in fp64.

Bounds, per output element, from the arithmetic: products of bf16 or fp32
operands summed over n terms in fp32 are off by at most n * 2^-23 * sum|a b|
(n additions and, for fp32 operands, n products, each within 2^-24 of a
partial sum); an activation moves an error by at most its slope (below 1.13
for each here) and is itself evaluated to 16 ulp; the result is rounded once
(bf16 2^-8, fp32 2^-24 of the value).  In the backward pass dz is rounded to
bf16 once before the products.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SLOPE = 1.13
EVAL = 16 * 2.0 ** -24
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]


def act64(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.relu(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    a, b = z.chunk(2, 1)
    return a * torch.sigmoid(a) * b


def pad(n, dtype):
    q = 8 if dtype == "bf16" else 4
    return (n + q - 1) // q * q


def padded(rows, cols, dtype, extra=0, fill=float("nan"), lead=()):
    """[*lead, rows, cols] view over rows with a gap (holding NaN) behind each."""
    ld = pad(cols, dtype) + extra
    t = torch.full((*lead, rows, ld), fill, dtype=TD[dtype], device=DEV)
    return t, t[..., :cols], ld


def values(view, gen, scale=1.0):
    view.copy_(torch.empty(view.shape, dtype=torch.float64).normal_(0, scale, generator=gen))


class Problem:
    """One product with its inputs, outputs (pre-filled with NaN) and fp64 reference."""

    def __init__(self, rows, K, N, dtype="bf16", act="none", groups=None, gather_k=0, bias=False, residual=False,
                 save=True, grad=None, extra=0, seed=0):
        # groups: list of row counts (with gaps before / after allowed through `rows`)
        g = torch.Generator().manual_seed(seed)
        self.rows, self.K, self.N, self.dtype, self.act = rows, K, N, dtype, act
        self.grad = grad or dtype
        E = len(groups) if groups is not None else 1
        self.E, self.groups, self.k = E, groups, gather_k
        self.oc = N // 2 if act == "swiglu" else N
        if groups is not None:
            off = torch.zeros(E + 1, dtype=torch.int32)
            off[1:] = torch.tensor(groups).cumsum(0)
            self.off_h = off.tolist()
            self.off = off.to(DEV)
            assert self.off_h[-1] <= rows
        else:
            self.off_h, self.off = [0, rows], None
        self.x_rows = rows
        self.pairs = None
        src = torch.arange(rows)
        if gather_k:
            self.x_rows = (rows + gather_k - 1) // gather_k
            pairs = torch.randperm(self.x_rows * gather_k, generator=g)[:rows].to(torch.int32)
            self.pairs = pairs.to(DEV)
            src = (pairs // gather_k).long()
        self.src = src
        self.xb, self.x, ldx = padded(self.x_rows, K, dtype, extra)
        values(self.x, g)
        self.wb, self.w, ldw = padded(N, K, dtype, extra, lead=(E,))
        values(self.w, g, K ** -0.5)
        self.bias = torch.empty(E, N).normal_(0, 0.5, generator=g).to(TD[dtype]).to(DEV) if bias else None
        self.yb, self.y, ldy = padded(rows, self.oc, dtype, extra)
        self.zb, self.z, ldz = padded(rows, N, dtype, extra)
        self.save = save
        self.res = None
        if residual:
            _, self.res, _ = padded(rows, self.oc, dtype, extra)
            values(self.res, g)
        _, self.dy, _ = padded(rows, self.oc, dtype, extra)
        values(self.dy, g)
        _, self.zin, _ = padded(rows, N, dtype, extra)
        values(self.zin, g, 1.5)
        self.dxb, self.dx, _ = padded(rows, K, dtype, extra)
        self.dwb, self.dw, _ = padded(N, K, self.grad, ldw - pad(K, self.grad), lead=(E,))
        self.dbias = torch.full((E, N), float("nan"), dtype=TD[self.grad], device=DEV)
        self.m = ds4.make_matmul(K, N, groups=E, dtype=dtype, act=act, grad=grad, ldx=ldx, ldw=ldw, ldy=ldy, ldz=ldz)

    def ws(self, backward):
        n = ds4.matmul_workspace_bytes(self.m, self.rows, backward)
        return torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) if n else None

    def forward(self, ws="own", stream=None):
        ws = self.ws(False) if isinstance(ws, str) else ws
        z = self.z if self.save else None
        if self.off is None:
            ds4.linear(self.m, self.rows, self.x, self.w, self.y, bias=self.bias, residual=self.res, z=z,
                       workspace=ws, stream=stream)
        else:
            ds4.grouped_matmul(self.m, self.rows, self.x, self.w, self.off, self.y, sorted_pair=self.pairs,
                               top_k=max(1, self.k), x_rows=self.x_rows, bias=self.bias, z=z, workspace=ws,
                               stream=stream)

    def backward(self, dx=True, dw=True, dbias=True, ws="own"):
        ws = self.ws(True) if isinstance(ws, str) else ws
        kw = dict(z=self.zin if self.act != "none" else None, dx=self.dx if dx else None,
                  dw=self.dw if dw else None, dbias=self.dbias if dbias else None, workspace=ws)
        x, w = (self.x if dw else None), (self.w if dx else None)
        if self.off is None:
            ds4.linear_backward(self.m, self.rows, x, w, self.dy, **kw)
        else:
            ds4.grouped_matmul_backward(self.m, self.rows, x, w, self.off, self.dy, sorted_pair=self.pairs,
                                        top_k=max(1, self.k), x_rows=self.x_rows, **kw)

    def check_forward(self):
        h, worst = HALF[self.dtype], 0.0
        x, w = self.x.double()[self.src.to(DEV)], self.w.double()
        for e in range(self.E):
            a, b = self.off_h[e], self.off_h[e + 1]
            if a == b:
                continue
            z = x[a:b] @ w[e].t()
            S = x[a:b].abs() @ w[e].abs().t()
            if self.bias is not None:
                z = z + self.bias[e].double()
                S = S + self.bias[e].double().abs()
            ez = (self.K + 1) * 2.0 ** -23 * S
            if self.save:
                worst = max(worst, self._cmp("z", self.z[a:b], z, ez + h * (z.abs() + ez)))
            y = act64(z, self.act)
            if self.act == "swiglu":
                g, u = z.chunk(2, 1)
                eg, eu = ez.chunk(2, 1)
                ey = SLOPE * eg * (u.abs() + eu) + act64(g, "silu").abs() * eu
            else:
                ey = SLOPE * ez
            ey = ey + EVAL * y.abs()
            if self.res is not None:
                y = y + self.res[a:b].double()
                ey = ey + 2.0 ** -24 * (y.abs() + ey)
            worst = max(worst, self._cmp("y", self.y[a:b], y, ey + h * (y.abs() + ey) + 1e-37))
        self._gaps(self.yb, self.oc)
        if self.save:
            self._gaps(self.zb, self.N)
        self._outside(self.y)
        return worst

    def check_backward(self, dx=True, dw=True, dbias=True):
        h, hg = HALF[self.dtype], HALF[self.grad]
        x, w = self.x.double()[self.src.to(DEV)], self.w.double()
        for e in range(self.E):
            a, b = self.off_h[e], self.off_h[e + 1]
            dy = self.dy[a:b].double()
            dz = dy
            if self.act != "none":
                z = self.zin[a:b].double().requires_grad_()
                dz, = torch.autograd.grad(act64(z, self.act), z, dy)
                dz = dz.detach()
            # evaluation of act' (its terms cancel: bounded by dy and, for SwiGLU, the factors)
            if self.act == "none":
                ev = torch.zeros_like(dz)
            elif self.act == "swiglu":
                g, u = self.zin[a:b].double().chunk(2, 1)
                ev = EVAL * torch.cat([dy * u * (1 + g.abs()), dy * g], 1).abs()
            else:
                ev = EVAL * (dy * (1 + self.zin[a:b].double().abs()) ** 2).abs()
            edz = ev + (h * dz.abs() if self.act != "none" else 0)
            if dx and b > a:
                r = dz @ w[e]
                S = dz.abs() @ w[e].abs()
                er = edz @ w[e].abs() + (self.N + 1) * 2.0 ** -23 * S
                self._cmp("dx", self.dx[a:b], r, er + h * (r.abs() + er))
            if dw:
                r = dz.t() @ x[a:b]
                S = dz.abs().t() @ x[a:b].abs()
                er = edz.t() @ x[a:b].abs() + (b - a + 1) * 2.0 ** -23 * S
                self._cmp("dw", self.dw[e], r, er + hg * (r.abs() + er))
            if dbias:
                r = dz.sum(0)
                er = ev.sum(0) + (b - a + 70) * 2.0 ** -24 * dz.abs().sum(0)
                self._cmp("dbias", self.dbias[e], r, er + hg * (r.abs() + er))
        if dx:
            self._gaps(self.dxb, self.K)
            self._outside(self.dx)
        if dw:
            self._gaps(self.dwb, self.K)

    def _cmp(self, name, got, ref, bound):
        got = got.double()
        assert torch.isfinite(got).all(), name
        r = ((got - ref).abs() - bound).max().item()
        assert r <= 0, (name, r, (got - ref).abs().max().item(), bound.max().item())
        return ((got - ref).abs() / bound.clamp(min=1e-300)).max().item()

    def _gaps(self, base, cols):
        assert torch.isnan(base[..., cols:].float()).all(), "written behind a row's end"

    def _outside(self, view):
        """Rows behind the last group (and before the first) keep what they held."""
        assert torch.isnan(view[self.off_h[-1]:].float()).all()


DENSE = [
    # rows, K, N: one row to long, odd sizes, tile borders
    (1, 1, 1), (1, 64, 16), (1, 1000, 333), (2, 7, 130), (3, 2048, 512), (5, 40, 48), (16, 513, 257), (17, 256, 96),
    (33, 96, 17), (64, 64, 64), (65, 65, 65), (100, 321, 259), (128, 128, 256), (129, 72, 514), (200, 1024, 320),
    (257, 200, 128), (300, 63, 600), (513, 520, 260),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,N", DENSE)
def test_linear_forward_sizes(rows, K, N, dtype):
    print(f"linear {rows}x{K}->{N} {dtype}", flush=True)
    p = Problem(rows, K, N, dtype, "none", bias=True, residual=rows % 2 == 0, seed=rows + K, extra=8 * (rows % 3))
    p.forward()
    p.check_forward()


@pytest.mark.parametrize("rows", [1, 7, 40, 150])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_linear_forward_acts(act, dtype, rows):
    for bias, res, save in ((True, True, True), (False, False, False)):
        print(f"linear {act} {dtype} rows={rows} bias={bias}", flush=True)
        p = Problem(rows, 136, 198, dtype, act, bias=bias, residual=res, save=save, seed=3 + rows)
        p.forward()
        p.check_forward()


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,K,N", DENSE)
def test_linear_backward_sizes(rows, K, N, dtype, grad):
    print(f"linear backward {rows}x{K}->{N} {dtype} {grad}", flush=True)
    p = Problem(rows, K, N, dtype, "none", grad=grad, seed=rows + N, extra=8 * (rows % 2))
    p.backward()
    p.check_backward()


@pytest.mark.parametrize("dtype,grad", [("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_acts(act, dtype, grad):
    for rows, K, N in ((1, 70, 34), (77, 136, 198), (400, 96, 272)):
        print(f"linear backward {act} {dtype} rows={rows}", flush=True)
        p = Problem(rows, K, N, dtype, act, grad=grad, seed=9 + rows)
        p.backward()
        p.check_backward()


@pytest.mark.parametrize("which", ["dx", "dw", "dbias"])
def test_linear_backward_one_output(which):
    p = Problem(90, 136, 198, "bf16", "silu", seed=4)
    want = {w: w == which for w in ("dx", "dw", "dbias")}
    p.backward(**want)
    p.check_backward(**want)
    torch.cuda.synchronize()
    for w, on in want.items():
        if not on:
            assert torch.isnan(getattr(p, w).float()).all(), w


GROUPS = [
    # rows of each expert: none, one, ragged, all in one, borders of a tile
    [1], [0], [0, 0, 5], [1, 0, 1, 1], [3, 130, 0, 64, 1], [0, 300, 0], [128, 256, 127, 129], [16, 17, 15, 1, 0, 33],
    [1] * 40, [0] * 30 + [2] + [0] * 30,
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("groups", GROUPS, ids=lambda g: "-".join(map(str, g))[:30])
def test_grouped(groups, dtype):
    for K, N, act, k in ((136, 264, "swiglu", 3), (264, 136, "none", 0), (77, 51, "gelu", 2)):
        rows = sum(groups) + (5 if len(groups) % 2 else 0)
        print(f"grouped {groups[:8]} {K}->{N} {act} {dtype}", flush=True)
        p = Problem(max(1, rows), K, N, dtype, act, groups=groups, gather_k=k, bias=True, seed=len(groups))
        p.forward()
        p.check_forward()
        p.backward()
        p.check_backward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_residual_in_place(dtype):
    """y may be the residual itself."""
    for rows in (1, 9, 200):
        p = Problem(rows, 128, 96, dtype, "silu", bias=True, residual=True, seed=6)
        keep = p.res.clone()
        p.y = p.res
        p.yb = torch.full((1, 97), float("nan"), device=DEV)
        p.forward()
        got = p.y.clone()
        p.res, p.y = keep, got
        p.save = False
        p.check_forward()


def test_gradients_against_differences():
    """dx, dw and dbias of sum(y * dy) by central differences of the forward pass in fp32 mode.

    Along a direction z moves by v per unit (z is linear in x, in w and in the bias).  The difference quotient over
    +-eps then differs from the derivative by
      - eps^2 / 6 * |dy| * |third derivative along v| per output: at most 2 |v|^3 for silu and both gelus, and for
        SwiGLU 0.5 |v_g|^3 |u| + 1.5 v_g^2 |v_u| (silu's second and third derivatives stay within 0.5), with u up to
        eps |v_u| further on;
      - at most |dy| |v| where z is within eps |v| of relu's kink;
      - the forward pass's own error, |dy| * (K + 20) * 2^-23 * (sum |x w| + |bias|) * 1.13 (SwiGLU: times 1 + |g| +
        |u|) on either side, over eps."""
    rows, K, N = 24, 20, 12
    eps = 2.0 ** -7
    for act in ACTS:
        p = Problem(rows, K, N, "f32", act, groups=[10, 0, 14], bias=True, seed=12)
        p.forward()
        p.zin = p.z.clone()
        p.backward()

        def loss():
            p.forward()
            return (p.y.double() * p.dy.double()).sum().item(), p.z.double()

        S = torch.cat([p.x[p.src.to(DEV)][a:b].double().abs() @ p.w[e].double().abs().t() + p.bias[e].double().abs()
                       for e, (a, b) in enumerate(((0, 10), (10, 10), (10, 24)))])
        dy, z = p.dy.double().abs(), p.zin.double()
        g = torch.Generator().manual_seed(2)
        for t, grad in ((p.x, p.dx), (p.w, p.dw), (p.bias, p.dbias)):
            d = torch.empty(t.shape).normal_(generator=g).to(DEV)
            t0 = t.clone()
            t.copy_(t0 + eps * d)
            up, zu = loss()
            t.copy_(t0 - eps * d)
            dn, zd = loss()
            t.copy_(t0)
            v = (zu - zd).abs() / (2 * eps)
            noise = (K + 20) * 2.0 ** -23 * (S + eps * v) * 1.13
            kink = dy * v * (z.abs() <= eps * v + 2 * noise) if act == "relu" else torch.zeros_like(v)
            if act == "swiglu":
                (vg, vu), (zg, zl) = v.chunk(2, 1), z.abs().chunk(2, 1)
                curve = 0.5 * vg ** 3 * (zl + eps * vu) + 1.5 * vg ** 2 * vu
                noise = sum(noise.chunk(2, 1)) * (1 + zg + zl)
            else:
                curve = 0 * v if act in ("none", "relu") else 2 * v ** 3
            tol = (dy * (eps ** 2 / 6 * curve + 2 * noise / eps)).sum().item() + kink.sum().item()
            want = (grad.double() * d.double()).sum().item()
            assert abs((up - dn) / (2 * eps) - want) <= tol, (act, want, (up - dn) / (2 * eps), tol)


def test_expert_layer_of_products():
    """An MoE layer with bf16 experts as it would be used: route, permute, gate/up products with SwiGLU through
    sorted_pair, down products, combine; then the whole backward pass with combine summing the token rows."""
    T, H, F, E, k = 150, 256, 128, 8, 2
    g = torch.Generator().manual_seed(1)
    cfg = ds4.make_config(H, F, E, k)
    bf = torch.bfloat16
    x = torch.empty(T, H).normal_(generator=g).to(bf).to(DEV)
    wu = torch.empty(E, 2 * F, H).normal_(0, H ** -0.5, generator=g).to(bf).to(DEV)
    wd = torch.empty(E, H, F).normal_(0, F ** -0.5, generator=g).to(bf).to(DEV)
    logits = torch.empty(T, E).normal_(generator=g).to(DEV)
    dy = torch.empty(T, H).normal_(generator=g).to(bf).to(DEV)
    P = T * k
    i32 = dict(dtype=torch.int32, device=DEV)
    idx, tw = torch.empty(T, k, **i32), torch.empty(T, k, device=DEV)
    off, sp, pp, act = (torch.empty(n, **i32) for n in (E + 1, P, P, E + 1))
    ds4.route(cfg, T, logits, idx, tw)
    ds4.permute(cfg, T, idx, off, sp, pp, act)
    up = ds4.make_matmul(H, 2 * F, groups=E, act="swiglu", grad="f32")
    dn = ds4.make_matmul(F, H, groups=E, grad="f32")
    ws = torch.empty(max(ds4.matmul_workspace_bytes(m, P, True) for m in (up, dn)), dtype=torch.uint8, device=DEV)
    h, z = torch.empty(P, F, dtype=bf, device=DEV), torch.empty(P, 2 * F, dtype=bf, device=DEV)
    eo, y = torch.empty(P, H, dtype=bf, device=DEV), torch.empty(T, H, dtype=bf, device=DEV)
    ds4.grouped_matmul(up, P, x, wu, off, h, sorted_pair=sp, top_k=k, z=z, workspace=ws)
    ds4.grouped_matmul(dn, P, h, wd, off, eo, workspace=ws)
    ds4.combine(cfg, T, eo, pp, tw, None, y)
    # backward: the gradient of a sorted row is its weight times its token's dy
    deo = (tw.view(-1)[sp.long()][:, None] * dy.float()[(sp // k).long()]).to(bf)
    dh, dxr = torch.empty_like(h), torch.empty(P, H, dtype=bf, device=DEV)
    dwu, dwd = torch.empty(wu.shape, device=DEV), torch.empty(wd.shape, device=DEV)
    dx = torch.empty_like(x)
    ds4.grouped_matmul_backward(dn, P, h, wd, off, deo, dx=dh, dw=dwd, workspace=ws)
    ds4.grouped_matmul_backward(up, P, x, wu, off, dh, z=z, sorted_pair=sp, top_k=k, dx=dxr, dw=dwu, workspace=ws)
    ds4.combine(cfg, T, dxr, pp, torch.ones_like(tw), None, dx)
    torch.cuda.synchronize()

    # the same layer in fp64 with autograd, for the same routing
    xd, wud, wdd = (t.double().requires_grad_() for t in (x, wu, wd))
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for j in range(k):
        for e in range(E):
            t = (idx[:, j] == e).nonzero()[:, 0]
            v = act64(xd[t] @ wud[e].t(), "swiglu") @ wdd[e].t()
            out = out.index_add(0, t, tw[t, j].double()[:, None] * v)
    out.backward(dy.double())

    def err(a, b):
        return ((a.double() - b).norm() / b.norm()).item()

    # each tensor passes at most five bf16 roundings (h, expert rows, deo, dh, dz, the result) of relative size up
    # to 2^-8 each; their joint effect on a norm is at most the sum
    for name, a, b in (("y", y, out.detach()), ("dx", dx, xd.grad), ("dwu", dwu, wud.grad), ("dwd", dwd, wdd.grad)):
        assert err(a, b) <= 6 * 2.0 ** -8, (name, err(a, b))


def test_deterministic_and_other_stream():
    p = Problem(300, 264, 200, "bf16", "gelu", groups=[100, 0, 150, 50], gather_k=2, bias=True, seed=21)
    p.forward()
    p.backward()
    keep = [t.clone() for t in (p.y, p.z, p.dx, p.dw, p.dbias)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in (p.y, p.z, p.dx, p.dw, p.dbias):
        t.fill_(float("nan"))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.forward()
        p.backward()
    torch.cuda.synchronize()
    for a, b in zip(keep, (p.y, p.z, p.dx, p.dw, p.dbias)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [4, 260])
def test_graph_replays(rows):
    """Forward and backward captured together, replayed with new inputs, against eager calls."""
    p = Problem(rows, 264, 200, "bf16", "swiglu", groups=[rows // 2, 0, rows - rows // 2], gather_k=2, bias=True, seed=8)
    outs = lambda: (p.y, p.z, p.dx, p.dw, p.dbias)
    wf, wb = p.ws(False), p.ws(True)

    def both():
        p.forward(ws=wf)
        p.backward(ws=wb)

    xs = [torch.randn_like(p.x) for _ in range(3)]
    refs = []
    for x in xs:
        p.x.copy_(x)
        both()
        refs.append([t.clone() for t in outs()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for rep in range(6):
        p.x.copy_(xs[rep % 3])
        for t in outs():
            t.fill_(float("nan"))
        torch.randn(1000, device=DEV).sum().item()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs(), refs[rep % 3]):
            assert torch.equal(a, b), rep


def test_corrupt_offsets_and_pairs_stay_inside():
    """Offsets that do not ascend within the rows leave their expert without rows; pair ids outside the tokens read
    some row of x."""
    p = Problem(60, 136, 72, "bf16", "none", groups=[20, 20, 20], gather_k=2, seed=30)
    p.off.copy_(torch.tensor([0, 20, 10, 100], dtype=torch.int32))
    p.pairs[:3] = torch.tensor([-7, 1 << 30, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    p.forward()
    torch.cuda.synchronize()
    assert torch.isfinite(p.y[:20].float()).all()
    assert torch.isnan(p.y[20:].float()).all()


def test_far_rows():
    """Rows whose elements lie beyond 2^32 bytes of x, y and dx."""
    rows, K, N = 2 ** 19 + 3, 4104, 24
    m = ds4.make_matmul(K, N)
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    x[-2:].normal_()
    w = torch.randn(N, K, device=DEV).to(torch.bfloat16)
    y = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(16, ds4.matmul_workspace_bytes(m, rows, True)), dtype=torch.uint8, device=DEV)
    ds4.linear(m, rows, x, w, y, workspace=ws)
    ref = x[-2:].double() @ w.double().t()
    S = x[-2:].double().abs() @ w.double().abs().t()
    assert ((y[-2:].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + K * 2.0 ** -22 * S).all()
    assert (y[:-2] == 0).all()
    dx = torch.full((rows, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    ds4.linear_backward(m, rows, None, w, y, dx=dx, workspace=ws)
    ref = y[-2:].double() @ w.double()
    S = y[-2:].double().abs() @ w.double().abs()
    assert ((dx[-2:].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + N * 2.0 ** -22 * S).all()
    assert (dx[:-2] == 0).all()


def test_wrong_device_is_refused():
    m = ds4.make_matmul(64, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    y = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ds4.Ds4MoeError) as ei:
        ds4.linear(m, 4, x, y, y)
    assert ei.value.status == -1


@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("K", [128, 520, 1031, 2100])
def test_few_rows(rows, K):
    """Decoding's sizes: contractions shorter and longer than a workgroup's waves share, with every epilogue."""
    for N, act in ((40, "none"), (272, "swiglu"), (34, "swiglu"), (1000, "gelu")):
        p = Problem(rows, K, N, "bf16", act, bias=True, residual=True, seed=rows + K)
        p.forward()
        p.check_forward()


@pytest.mark.parametrize("mode", ["forward", "dx", "dw"])
def test_split_contraction(mode):
    """Few outputs over a long contraction: partial sums of its splits, joined in order, the same every time."""
    for rows, K, N, groups in ((40, 4104, 72, None), (100, 8192, 130, None), (60, 2056, 264, [30, 0, 25]),
                               (4100, 72, 40, None), (70, 96, 4104, None), (3000, 40, 136, [1500, 3, 1497])):
        print(f"split {mode} {rows}x{K}->{N}", flush=True)
        p = Problem(rows, K, N, "bf16", "swiglu", groups=groups, bias=True, seed=K)
        if mode == "forward":
            p.forward()
            p.check_forward()
            first = p.y.clone()
            p.forward()
            assert torch.equal(first[: p.off_h[-1]], p.y[: p.off_h[-1]])
        else:
            want = {w: w == mode for w in ("dx", "dw", "dbias")}
            p.backward(**want)
            p.check_backward(**want)


def test_wide_head_few_rows():
    """A head wide enough that 16 rows take the tiles and 3 rows the streaming kernel."""
    for rows in (3, 16):
        p = Problem(rows, 264, 33000, "bf16", "none", seed=rows, save=False)
        p.forward()
        p.check_forward()


def test_one_group_of_many_chunks():
    """A group's rows beyond what one thread of the plan lists by itself."""
    p = Problem(5003, 72, 40, "bf16", "relu", groups=[2, 4990, 0, 7], gather_k=2, bias=True, seed=5)
    p.forward()
    p.check_forward()
    p.backward()
    p.check_backward()


def test_two_streams_at_once():
    """Calls on two streams with their own outputs and workspaces."""
    ps = [Problem(260, 264, 200, "bf16", "swiglu", groups=[130, 0, 130], gather_k=2, bias=True, seed=s) for s in (1, 2)]
    refs = []
    for p in ps:
        p.forward()
        p.backward()
        refs.append([t.clone() for t in (p.y, p.z, p.dx, p.dw, p.dbias)])
    ws = [(p.ws(False), p.ws(True)) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s, (wf, wb) in zip(ps, streams, ws):
            with torch.cuda.stream(s):
                p.forward(ws=wf)
                p.backward(ws=wb)
    torch.cuda.synchronize()
    for p, r in zip(ps, refs):
        for a, b in zip((p.y, p.z, p.dx, p.dw, p.dbias), r):
            assert torch.equal(a, b)


def test_offsets_that_start_behind_zero_and_one_group():
    """One group of part of the rows: the others are left as they were."""
    for dtype in ("bf16", "f32"):
        for rows, a, b in ((12, 3, 9), (300, 17, 290)):
            p = Problem(rows, 72, 40, dtype, "silu", groups=[rows], bias=True, seed=rows)
            p.off.copy_(torch.tensor([a, b], dtype=torch.int32))
            p.off_h = [a, b]
            p.forward()
            p.check_forward()
            p.backward()
            p.check_backward()
            assert torch.isnan(p.y[:a].float()).all() and torch.isnan(p.dx[:a].float()).all()


# sizes that between them take every tile shape in every direction (and split contractions), with ragged ends
@pytest.mark.parametrize("rows,K,N", [(2045, 2050, 7170), (4090, 7162, 2042), (1021, 1026, 7170), (700, 1026, 5000)])
def test_large_linear_shapes(rows, K, N):
    print(f"large {rows}x{K}->{N}", flush=True)
    p = Problem(rows, K, N, "bf16", "swiglu", bias=True, residual=True, seed=rows)
    p.forward()
    p.check_forward()
    p.backward()
    p.check_backward()
    del p
    p = Problem(rows, K, N, "bf16", "gelu", grad="f32", save=False, seed=rows + 1)
    p.forward()
    p.check_forward()
    p.backward(dbias=False)
    p.check_backward(dbias=False)


@pytest.mark.parametrize("groups", [[2600, 0, 1, 3000, 900, 1100, 30, 369], [1] * 3 + [0, 700, 150, 260, 5] * 3 + [90] * 7 +
                                    [0, 10, 1], [200] * 7 + [100]], ids=["few", "many", "even"])
def test_large_grouped_shapes(groups):
    rows = sum(groups) + 11
    print(f"large grouped {len(groups)} groups, {rows} rows", flush=True)
    p = Problem(rows, 1026, 2042, "bf16", "silu", groups=groups, gather_k=3, bias=True, seed=rows)
    p.forward()
    p.check_forward()
    p.backward()
    p.check_backward()
    del p
    p = Problem(rows, 1026, 2042, "bf16", "none", groups=groups, grad="f32", save=False, seed=rows)
    p.forward()
    p.check_forward()
    p.backward()
    p.check_backward()
