"""Rows by expert and back (ds4moe_dispatch, ds4moe_collect, their gradients,
ds4moe_route_backward) against the formulas in fp64.

Bounds, per output element, from the arithmetic: an unweighted row is copied
exactly; a weighted one takes one fp32 product (2^-24) and the result's rounding
(bf16 2^-8, fp32 2^-24 of the value).  A sum of n products in fp32 is off by at
most n * 2^-23 * sum|a b| (n products and n additions, each within 2^-24 of a
partial sum of absolute values), then rounded once.  dlogits = w (dw - s) with s
a sum of k products: its error is at most 2^-23 * |w| * ((k + 2) * sum_i |w_i dw_i| + 2 |dw|).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
QUANT = {"bf16": 8, "f32": 4}


def matrix(rows, cols, dtype, gen=None, gap=0):
    """View of rows that start at 16-byte boundaries, NaN in the gaps behind them (and, without gen, everywhere)."""
    q = QUANT[dtype]
    ld = (cols + q - 1) // q * q + gap * q
    buf = torch.full((rows, ld), float("nan"), dtype=TD[dtype], device=DEV)
    if gen is not None:
        buf[:, :cols] = torch.empty(rows, cols, dtype=torch.float64).normal_(0, 1, generator=gen).to(TD[dtype]).to(DEV)
    return buf, buf[:, :cols], ld


class Case:
    def __init__(self, T, k, H, dtype="bf16", weighted=True, layout="sorted", gap=0, E=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.k, self.H, self.dtype = T, k, H, dtype
        P = T * k
        if layout == "sorted":
            self.rows = P
            pos = torch.randperm(P, generator=g)
        else:   # more or fewer rows than pairs, any of them empty, about a third of the pairs dropped
            self.rows = max(1, P + 3 if layout == "roomy" else (2 * P) // 3)
            pos = torch.randperm(max(self.rows, P), generator=g)[:P]
            pos[torch.rand(P, generator=g) < 0.2] = -1
            pos[pos >= self.rows] = self.rows + 5
        self.pos_h = pos
        inv = torch.full((self.rows,), -1, dtype=torch.int64)
        ok = (pos >= 0) & (pos < self.rows)
        inv[pos[ok]] = torch.arange(P)[ok]
        inv[(inv < 0) & (torch.rand(self.rows, generator=g) < 0.5)] = P + 7     # both ends name no pair
        self.ok = ok.to(DEV)
        self.inv = inv.to(DEV)
        self.pos = pos.to(torch.int32).to(DEV)
        self.sorted_pair = inv.to(torch.int32).to(DEV)
        w = torch.empty(T, k, dtype=torch.float32).uniform_(-1, 1, generator=g)
        w.view(-1)[~ok] = float("nan")      # a dropped pair's weight is never used
        self.w = w.to(DEV) if weighted else None
        w1 = w if weighted else torch.ones(T, k)
        self.w64 = torch.where(ok.view(T, k), w1.double(), torch.zeros(T, k, dtype=torch.float64)).to(DEV)
        self.tok_buf, self.tok, ldx = matrix(T, H, dtype, g, gap)
        self.row_buf, self.row, ldr = matrix(self.rows, H, dtype, g, 2 * gap)
        self.row[self.inv.clamp(max=P) % (P + 1) == P] = float("nan")           # rows without a pair are never read
        self.row[self.inv < 0] = float("nan")
        self.base_buf, self.base, _ = matrix(T, H, dtype, g, gap)
        self.d = ds4.make_rows(H, k, dtype, ldx=ldx, ldr=ldr)
        self.gap = gap

    def pairs64(self):
        """[T, k, H] of the pairs' rows, 0 for dropped pairs."""
        p = self.row.double()[self.pos.long().clamp(0, self.rows - 1)]
        return torch.where(self.ok[:, None], p, torch.zeros((), dtype=torch.float64, device=DEV)).view(self.T, self.k, self.H)

    def check_rows(self, buf, got, before, zeros):
        """w * tok at the pairs' rows; zeros or what was there at the others; gaps untouched."""
        p = self.inv
        has = (p >= 0) & (p < self.T * self.k)
        want = self.tok.double()[(p[has] // self.k)] * self.w64.view(-1)[p[has]][:, None]
        err = (got[has].double() - want).abs()
        if self.w is None:
            assert torch.equal(got[has].double(), want)
        else:
            assert (err <= (HALF[self.dtype] + 2.0 ** -23) * want.abs() + 1e-40).all()
        if zeros:
            assert (got[~has] == 0).all()
        else:
            assert torch.equal(got[~has], before[~has]) or (got[~has].isnan() == before[~has].isnan()).all()
        assert buf[:, self.H:].isnan().all()

    def check_sums(self, buf, got, base):
        p = self.pairs64() * self.w64[:, :, None]
        want, size = p.sum(1), p.abs().sum(1)
        if base is not None:
            want, size = want + base.double(), size + base.double().abs()
        tol = (self.k + 1) * 2.0 ** -23 * size + HALF[self.dtype] * want.abs() + 1e-40
        assert ((got.double() - want).abs() <= tol).all()
        assert buf[:, self.H:].isnan().all()

    def check_dots(self, got):
        p = self.pairs64()
        v = self.tok.double()[:, None]
        want, size = (p * v).sum(2), (p * v).abs().sum(2)
        assert ((got.double() - want).abs() <= self.H * 2.0 ** -23 * size).all()
        assert (got.view(-1)[~self.ok] == 0).all()


SIZES = [(1, 1, 1), (1, 8, 7168), (3, 2, 7), (5, 3, 459), (16, 8, 7168), (2, 64, 130), (33, 5, 1024), (300, 7, 2050),
         (7, 15, 4099), (1, 3, 20000), (700, 1, 64), (257, 12, 515)]


@pytest.mark.parametrize("layout", ["sorted", "roomy", "tight"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,H", SIZES)
def test_all_directions(T, k, H, dtype, layout):
    for weighted, gap in ((True, 0), (False, 1), (True, 3)):
        c = Case(T, k, H, dtype, weighted, layout, gap, seed=T + k + H)
        for zeros in (False, True):
            sp = c.sorted_pair if zeros else None
            buf, out, _ = matrix(c.rows, H, dtype, None, 2 * gap)
            ds4.dispatch(c.d, T, c.rows, c.tok, c.pos, out, topk_w=c.w, sorted_pair=sp)
            c.check_rows(buf, out, torch.full_like(out, float("nan")), zeros)
            buf, out, _ = matrix(c.rows, H, dtype, None, 2 * gap)
            dw = torch.full((T, k), float("nan"), device=DEV)
            ds4.collect_backward(c.d, T, c.rows, c.tok, c.pos, expert_rows=c.row, topk_w=c.w, sorted_pair=sp, drows=out,
                                 dtopk_w=dw)
            c.check_rows(buf, out, torch.full_like(out, float("nan")), zeros)
            c.check_dots(dw)
        for base in (None, c.base):
            buf, y, _ = matrix(T, H, dtype, None, gap)
            ds4.collect(c.d, T, c.rows, c.row, c.pos, y, topk_w=c.w, base=base)
            c.check_sums(buf, y, base)
        buf, dx, _ = matrix(T, H, dtype, None, gap)
        dw = torch.full((T, k), float("nan"), device=DEV)
        ds4.dispatch_backward(c.d, T, c.rows, c.row, c.pos, topk_w=c.w, x=c.tok, dx=dx, dtopk_w=dw)
        c.check_sums(buf, dx, None)
        c.check_dots(dw)


def test_one_output_alone():
    c = Case(40, 6, 900, "bf16", layout="roomy", seed=3)
    dw = torch.full((3, 40, 6), float("nan"), device=DEV)
    ds4.collect_backward(c.d, 40, c.rows, c.tok, c.pos, expert_rows=c.row, topk_w=c.w, dtopk_w=dw[0])
    ds4.dispatch_backward(c.d, 40, c.rows, c.row, c.pos, topk_w=c.w, x=c.tok, dtopk_w=dw[1])
    ds4.collect_backward(c.d, 40, c.rows, c.tok, c.pos, expert_rows=c.row, dtopk_w=dw[2], sorted_pair=c.sorted_pair)
    for i in range(3):
        c.check_dots(dw[i])
    buf, out, _ = matrix(c.rows, 900, "bf16")
    ds4.collect_backward(c.d, 40, c.rows, c.tok, c.pos, topk_w=c.w, drows=out)
    c.check_rows(buf, out, torch.full_like(out, float("nan")), False)
    buf, dx, _ = matrix(40, 900, "bf16")
    ds4.dispatch_backward(c.d, 40, c.rows, c.row, c.pos, topk_w=c.w, dx=dx)
    c.check_sums(buf, dx, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(dtype):
    """y over base, and the rows' gradients over the rows themselves."""
    c = Case(65, 4, 1300, dtype, layout="roomy", seed=5)
    base = c.base_buf.clone()
    y = base[:, :1300]
    ds4.collect(c.d, 65, c.rows, c.row, c.pos, y, topk_w=c.w, base=y)
    c.check_sums(base, y, c.base)
    rows = c.row_buf.clone()
    dw = torch.full((65, 4), float("nan"), device=DEV)
    ds4.collect_backward(c.d, 65, c.rows, c.tok, c.pos, expert_rows=rows[:, :1300], topk_w=c.w,
                         sorted_pair=c.sorted_pair, drows=rows[:, :1300], dtopk_w=dw)
    c.check_dots(dw)
    c.check_rows(rows, rows[:, :1300], None, True)


def test_infinities_stay_in_their_row():
    c = Case(20, 2, 256, "f32", layout="sorted", seed=6)
    c.row[5, 17] = float("inf")
    c.row[9, 3] = float("nan")
    y = torch.empty(20, 256, device=DEV)
    ds4.collect(c.d, 20, c.rows, c.row, c.pos, y, topk_w=c.w)
    bad = torch.zeros(20, 256, dtype=torch.bool, device=DEV)
    bad[c.inv[5] // 2, 17] = True
    bad[c.inv[9] // 2, 3] = True
    assert torch.equal(~torch.isfinite(y), bad)


@pytest.mark.parametrize("which", ["to rows", "to tokens"])
def test_far_rows(which):
    """Rows whose elements lie more than 2^31 elements into their tensor."""
    H, k = 8192, 2
    rows = (1 << 18) + 40
    T = 8
    buf = torch.empty(rows, H, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(1)
    pos = torch.tensor([0, rows - 1, rows - 2, 3, 1 << 18, (1 << 18) + 1, 5, -1, 7, 9, rows, 11, 12, 13, rows - 9, 2],
                       dtype=torch.int32)
    d = ds4.make_rows(H, k)
    x = torch.empty(T, H).normal_(generator=g).bfloat16().to(DEV)
    at = pos.long().to(DEV)
    ok = (at >= 0) & (at < rows)
    if which == "to rows":
        buf[at[ok]] = 0
        ds4.dispatch(d, T, rows, x, pos.to(DEV), buf)
        assert torch.equal(buf[at[ok]], x[torch.arange(16, device=DEV)[ok] // 2])
    else:
        vals = torch.empty(16, H).normal_(generator=g).bfloat16().to(DEV)
        buf[at[ok]] = vals[ok]
        y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        ds4.collect(d, T, rows, buf, pos.to(DEV), y)
        want = torch.where(ok[:, None], vals.double(), 0.0).view(T, 2, H).sum(1)
        assert ((y.double() - want).abs() <= HALF["bf16"] * want.abs() + 2.0 ** -22 * vals.double().abs().view(T, 2, H).sum(1)).all()


@pytest.mark.parametrize("layout", ["sorted", "roomy"])
def test_rows_that_no_cache_holds(layout):
    """Rows of more than 256 MB, which are stored another way."""
    T, k, H = 4100, 8, 4104
    c = Case(T, k, H, "bf16", layout=layout, seed=21)
    for zeros in (False, True):
        sp = c.sorted_pair if zeros else None
        buf, out, _ = matrix(c.rows, H, "bf16")
        ds4.dispatch(c.d, T, c.rows, c.tok, c.pos, out, topk_w=c.w, sorted_pair=sp)
        c.check_rows(buf, out, torch.full_like(out, float("nan")), zeros)
    rows, dw = c.row_buf.clone(), torch.empty(T, k, device=DEV)
    ds4.collect_backward(c.d, T, c.rows, c.tok, c.pos, expert_rows=rows[:, :H], topk_w=c.w, sorted_pair=c.sorted_pair,
                         drows=rows[:, :H], dtopk_w=dw)
    c.check_rows(rows, rows[:, :H], None, True)
    c.check_dots(dw)


@pytest.mark.parametrize("T,k,H,dtype", [(1 << 20, 1, 8, "bf16"), (2, 2, 1 << 20, "f32"), (3, 1, (1 << 20) - 3, "bf16"),
                                         (1 << 17, 8, 4, "f32")])
def test_limits(T, k, H, dtype):
    c = Case(T, k, H, dtype, layout="roomy", seed=22)
    buf, out, _ = matrix(c.rows, H, dtype)
    ds4.dispatch(c.d, T, c.rows, c.tok, c.pos, out, topk_w=c.w, sorted_pair=c.sorted_pair)
    c.check_rows(buf, out, None, True)
    buf, dx, _ = matrix(T, H, dtype)
    dw = torch.full((T, k), float("nan"), device=DEV)
    ds4.dispatch_backward(c.d, T, c.rows, c.row, c.pos, topk_w=c.w, x=c.tok, dx=dx, dtopk_w=dw)
    c.check_sums(buf, dx, None)
    c.check_dots(dw)


# ---- the router's gradient -----------------------------------------------------------

@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (5, 256, 8), (1, 1, 1), (67, 1024, 64), (300, 100, 7), (2, 65, 64)])
def test_route_backward(T, E, k):
    g = torch.Generator().manual_seed(T + E)
    cfg = ds4.make_config(256, 128, E, k)
    logits = torch.empty(T, E).normal_(0, 2, generator=g).to(DEV)
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, device=DEV)
    ds4.route(cfg, T, logits, idx, w)
    dw = torch.empty(T, k).normal_(generator=g).to(DEV)
    dl = torch.full((T, E), float("nan"), device=DEV)
    ds4.route_backward(cfg, T, idx, w, dw, dl)
    w64, d64 = w.double(), dw.double()
    s = (w64 * d64).sum(1, keepdim=True)
    want = torch.zeros(T, E, dtype=torch.float64, device=DEV).scatter_(1, idx.long(), w64 * (d64 - s))
    tol = 2.0 ** -23 * w64 * ((k + 2) * (w64 * d64).abs().sum(1, keepdim=True) + 2 * d64.abs())
    tol = torch.zeros(T, E, dtype=torch.float64, device=DEV).scatter_(1, idx.long(), tol)
    assert ((dl.double() - want).abs() <= tol).all()


def test_route_backward_skips_ids_outside():
    cfg = ds4.make_config(256, 128, 8, 3)
    idx = torch.tensor([[5, -1, 8], [0, 1, 1 << 30]], dtype=torch.int32, device=DEV)
    w = torch.full((2, 3), 1 / 3, device=DEV)
    dw = torch.tensor([[3.0, 0.0, 0.0], [0.0, 3.0, 0.0]], device=DEV)
    buf = torch.full((4, 8), 7.0, device=DEV)
    ds4.route_backward(cfg, 2, idx, w, dw, buf[1:3])
    assert (buf[0] == 7).all() and (buf[3] == 7).all()


def test_gradients_against_differences():
    """L = sum dy * collect(rows, softmax of the chosen logits), all in fp32: central differences of the calls
    themselves along random directions.  With |step| = h the difference's own error is about h^2 times the third
    derivative plus 2^-24 |L| / h; at h = 2^-6 and |L| about 100 both are below 0.02 of the gradients' size here."""
    T, E, k, H = 6, 12, 4, 40
    g = torch.Generator().manual_seed(8)
    cfg = ds4.make_config(256, 128, E, k)
    d = ds4.make_rows(H, k, "f32")
    logits = torch.empty(T, E).normal_(generator=g).to(DEV)
    rows = torch.empty(T * k, H).normal_(generator=g).to(DEV)
    dy = torch.empty(T, H).normal_(generator=g).to(DEV)
    pos = torch.randperm(T * k, generator=g).to(torch.int32).to(DEV)
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, device=DEV)
    y = torch.empty(T, H, device=DEV)

    def loss(lg, r):
        ds4.route(cfg, T, lg, idx, w)
        chosen = idx.clone()
        ds4.collect(d, T, T * k, r, pos, y, topk_w=w)
        return float((y.double() * dy.double()).sum()), chosen

    _, chosen = loss(logits, rows)
    drows, dw, dl = torch.empty_like(rows), torch.empty(T, k, device=DEV), torch.empty(T, E, device=DEV)
    ds4.collect_backward(d, T, T * k, dy, pos, expert_rows=rows, topk_w=w, drows=drows, dtopk_w=dw)
    ds4.route_backward(cfg, T, idx, w, dw, dl)
    h = 2.0 ** -6
    for seed in range(4):
        v = torch.empty(T, E).normal_(generator=g).to(DEV)
        v = torch.zeros_like(v).scatter_(1, chosen.long(), v.gather(1, chosen.long()))  # (the choice stays)
        r = torch.empty(T * k, H).normal_(generator=g).to(DEV)
        (a, ca), (b, cb) = loss(logits + h * v, rows + h * r), loss(logits - h * v, rows - h * r)
        if not (torch.equal(ca.sort(1).values, cb.sort(1).values) and torch.equal(ca.sort(1).values, chosen.sort(1).values)):
            continue
        if not (torch.equal(ca, chosen) and torch.equal(cb, chosen)):
            continue    # (a change of slots pairs other rows with the weights)
        want = float((dl.double() * v.double()).sum() + (drows.double() * r.double()).sum())
        size = float((dl.double() * v.double()).norm() + (drows.double() * r.double()).norm())
        assert abs((a - b) / (2 * h) - want) <= 0.02 * size


# ---- together --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_of_experts_forward_and_backward(dtype):
    """route, permute, dispatch, two grouped products, collect, and every gradient back to x, the weights and the
    logits, against fp64 autograd.  Intermediates are rounded to the rows' type, so errors are judged by norm: each of
    the at most 8 roundings along a path is below 2^-8 (bf16) or, with sums of up to 256 terms, 2^-16 (fp32)."""
    T, E, k, H, F = 70, 6, 3, 256, 128
    g = torch.Generator().manual_seed(9)
    t = TD[dtype]
    cfg = ds4.make_config(H, F, E, k)
    P = T * k
    mk = lambda *s, sc=1.0: torch.empty(*s).normal_(0, sc, generator=g).to(t).to(DEV)
    x, w1, w2, dy = mk(T, H), mk(E, F, H, sc=H ** -0.5), mk(E, H, F, sc=F ** -0.5), mk(T, H)
    logits = torch.empty(T, E).normal_(generator=g).to(DEV)
    idx, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    off, sp, pp, act = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (E + 1, P, P, E + 1))
    ds4.route(cfg, T, logits, idx, w)
    ds4.permute(cfg, T, idx, off, sp, pp, act)
    d = ds4.make_rows(H, k, dtype)
    m1, m2 = ds4.make_matmul(H, F, groups=E, dtype=dtype, act="silu"), ds4.make_matmul(F, H, groups=E, dtype=dtype)
    new = lambda *s: torch.empty(*s, dtype=t, device=DEV)
    ws = torch.empty(max(ds4.matmul_workspace_bytes(m, P, b) for m in (m1, m2) for b in (False, True)),
                     dtype=torch.uint8, device=DEV)
    xs, hz, hh, eo, y = new(P, H), new(P, F), new(P, F), new(P, H), new(T, H)
    ds4.dispatch(d, T, P, x, pp, xs)
    ds4.grouped_matmul(m1, P, xs, w1, off, hh, z=hz, workspace=ws)
    ds4.grouped_matmul(m2, P, hh, w2, off, eo, workspace=ws)
    ds4.collect(d, T, P, eo, pp, y, topk_w=w, base=x)
    deo, dh, dxs, dx, dw1, dw2 = new(P, H), new(P, F), new(P, H), new(T, H), torch.empty_like(w1), torch.empty_like(w2)
    dw, dl = torch.empty(T, k, device=DEV), torch.empty(T, E, device=DEV)
    ds4.collect_backward(d, T, P, dy, pp, expert_rows=eo, topk_w=w, drows=deo, dtopk_w=dw)
    ds4.route_backward(cfg, T, idx, w, dw, dl)
    ds4.grouped_matmul_backward(m2, P, hh, w2, off, deo, dx=dh, dw=dw2, workspace=ws)
    ds4.grouped_matmul_backward(m1, P, xs, w1, off, dh, z=hz, dx=dxs, dw=dw1, workspace=ws)
    ds4.dispatch_backward(d, T, P, dxs, pp, dx=dx)
    leaves = [v.double().cpu().requires_grad_() for v in (x, w1, w2, logits)]
    X, W1, W2, L = leaves
    I = idx.long().cpu()
    wt = torch.softmax(L.gather(1, I), 1)
    out = X
    for j in range(k):
        a = torch.nn.functional.silu(torch.einsum("th,tfh->tf", X, W1[I[:, j]]))
        out = out + wt[:, j:j + 1] * torch.einsum("tf,thf->th", a, W2[I[:, j]])
    out.backward(dy.double().cpu())
    tol = 8 * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -16)
    for name, got, want in (("y", y, out), ("dx", dx.double() + dy.double(), X.grad), ("dw1", dw1, W1.grad), ("dw2", dw2, W2.grad),
                            ("dlogits", dl, L.grad)):
        want = want.detach().to(DEV)
        assert float((got.double() - want).norm() / want.norm()) <= tol, name


def test_graph_replays_and_streams():
    c = Case(90, 8, 1500, "bf16", layout="roomy", seed=11)
    T, H = 90, 1500

    def bufs():
        return (matrix(c.rows, H, "bf16")[1], matrix(T, H, "bf16")[1], torch.empty(T, 8, device=DEV),
                matrix(c.rows, H, "bf16")[1], matrix(T, H, "bf16")[1], torch.empty(T, 8, device=DEV))

    def run(b, stream=None):
        ds4.dispatch(c.d, T, c.rows, c.tok, c.pos, b[0], topk_w=c.w, sorted_pair=c.sorted_pair, stream=stream)
        ds4.collect(c.d, T, c.rows, c.row, c.pos, b[1], topk_w=c.w, base=c.base, stream=stream)
        ds4.collect_backward(c.d, T, c.rows, c.tok, c.pos, expert_rows=c.row, topk_w=c.w, sorted_pair=c.sorted_pair,
                             drows=b[3], dtopk_w=b[2], stream=stream)
        ds4.dispatch_backward(c.d, T, c.rows, c.row, c.pos, topk_w=c.w, x=c.tok, dx=b[4], dtopk_w=b[5], stream=stream)

    want = bufs()
    run(want)
    a, b = bufs(), bufs()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    run(a, s1)
    run(b, s2)
    torch.cuda.synchronize()
    for o in (a, b):
        assert all(torch.equal(x, y) for x, y in zip(o, want))
    got = bufs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(got)
    for i in range(3):
        for t in got:
            t.fill_(float("nan"))
        c.tok.mul_(2.0)
        c.row.mul_(0.5)
        run(want)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
