"""Products in 8-bit integers (ds4moe_linear_int8, ds4moe_grouped_matmul_int8)
and the rows' quantization against their definitions in fp64.

Codes have to be equal.  Bounds of the products, per output element: the sum is
exact; its conversion to fp32, the two scales and the bias are four roundings of
at most 2^-24 of the values they take (|z| without the bias, and |bias|); an
activation moves an error by at most its slope (below 1.13 for each here) and is
itself evaluated to 16 ulp; SwiGLU multiplies two such values; the residual's
addition and the result's rounding (bf16 2^-8, fp32 2^-24) follow.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 2.0 ** -24
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]


# ---- quantization ----------------------------------------------------------------------

def reference_codes(x):
    """Codes and scale of rows in fp64: x * 127 is exact, and its quotient by top, both of at most 31 bits, lies on a
    whole number and a half or at least 2^-33 of it away, so fp64's division decides as the exact one does."""
    x = x.double()
    top = x.abs().amax(1)
    fine = torch.isfinite(top)
    q = torch.round(x * 127 / torch.where((top > 0) & fine, top, torch.ones_like(top))[:, None])
    q = torch.where(fine[:, None], q, torch.zeros_like(q)).to(torch.int8)
    scale = torch.where(fine, (top.float() / 127), torch.full_like(top.float(), float("nan")))
    return q, scale


def quantize_and_check(x, cols, gap=0):
    """x: [rows][>= cols] on the device, rows at 16-byte boundaries."""
    rows = x.shape[0]
    ldq = (cols + 15) // 16 * 16 + 16 * gap
    buf = torch.full((rows, ldq), 77, dtype=torch.int8, device=DEV)
    scale = torch.full((rows,), -5.0, device=DEV)
    ds4.quantize_rows_int8(rows, cols, x[:, :cols], buf[:, :cols], scale)
    q, s = reference_codes(x[:, :cols].cpu())
    assert torch.equal(buf[:, :cols].cpu(), q)
    assert torch.equal(scale.cpu().nan_to_num(nan=-1.0), s.nan_to_num(nan=-1.0))
    assert (buf[:, cols:] == 77).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7168), (3, 7), (5, 129), (9, 512), (6, 1024), (7, 2051), (4, 8192),
                                       (3, 8200), (2, 40000), (1000, 300), (2, 1 << 20)])
def test_quantize(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    for gap in (0, 1):
        ld = (cols + 7) // 8 * 8 + 8 * gap
        x = torch.full((rows, ld), float("nan"), dtype=TD[dtype])
        x[:, :cols] = torch.empty(rows, cols).normal_(generator=g).to(TD[dtype])
        x[:, :cols] *= torch.exp2(torch.randint(-60, 60, (rows, 1), generator=g).float()).to(TD[dtype])
        quantize_and_check(x.to(DEV), cols, gap)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_ties(dtype):
    """Every half between codes, at many scales: even whole numbers win."""
    x = torch.cat([torch.arange(-254, 255), torch.arange(-254, 255, 2)]).float()[None]      # top 254: code x / 2
    for e in range(-120, 120, 7):
        quantize_and_check((x * 2.0 ** e).to(TD[dtype]).to(DEV), x.shape[1] // 8 * 8)
    if dtype == "f32":      # neighbours of the halves
        v = torch.arange(-253, 254, 2).float()
        near = torch.cat([v, torch.nextafter(v, v + 9), torch.nextafter(v, v - 9), torch.tensor([254.0])])
        quantize_and_check(near[None, -760:].to(DEV), 760)
        odd = near / 3 * 1.1
        quantize_and_check(odd[None, -760:].to(DEV), 760)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_extremes(dtype):
    info = torch.finfo(TD[dtype])
    x = torch.zeros(12, 256, dtype=TD[dtype])
    g = torch.Generator().manual_seed(2)
    x[1] = info.max * torch.rand(256, generator=g)
    x[2] = info.tiny * torch.rand(256, generator=g)                # subnormal values
    x[3, 5] = info.tiny * 2.0 ** -5
    x[4, 9] = -info.max
    x[4, 10] = info.tiny
    x[5] = torch.randn(256, generator=g)
    x[5, 100] = float("inf")
    x[6] = torch.randn(256, generator=g)
    x[6, 255] = float("nan")
    x[7, 0] = float("-inf")
    x[8] = -0.0
    x[9] = -1.0
    x[10, 3] = 2.0 ** 64
    x[11, 3] = 2.0 ** -64
    quantize_and_check(x.to(DEV), 256)
    quantize_and_check(x.to(DEV), 250)


# ---- products ----------------------------------------------------------------------------

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


def codes(g, lead, cols, gap=0):
    """int8 codes, every byte among them, 99 in the gaps."""
    ld = (cols + 15) // 16 * 16 + 16 * gap
    t = torch.randint(-128, 128, (*lead, ld), generator=g, dtype=torch.int8)
    t[..., cols:] = 99
    return t.to(DEV)[..., :cols], ld


class Problem:
    def __init__(self, rows, K, N, dtype="bf16", act="none", groups=None, gather_k=0, bias=False, residual=False, gap=0,
                 seed=0):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.K, self.N, self.dtype, self.act, self.k = rows, K, N, dtype, act, gather_k
        E = len(groups) if groups is not None else 1
        self.oc = N // 2 if act == "swiglu" else N
        self.off_h, self.off = [0, rows], None
        if groups is not None:
            off = torch.zeros(E + 1, dtype=torch.int32)
            off[1:] = torch.tensor(groups).cumsum(0)
            self.off_h, self.off = off.tolist(), off.to(DEV)
        self.x_rows, self.pairs, self.src = rows, None, torch.arange(rows, device=DEV)
        if gather_k:
            self.x_rows = (rows + gather_k - 1) // gather_k
            pairs = torch.randperm(self.x_rows * gather_k, generator=g)[:rows].to(torch.int32)
            self.pairs, self.src = pairs.to(DEV), (pairs // gather_k).long().to(DEV)
        self.x, ldx = codes(g, (self.x_rows,), K, gap)
        self.w, ldw = codes(g, (E, N), K, 2 * gap)
        # z is of the order of 1
        self.xs = (torch.rand(self.x_rows, generator=g) + 0.5).to(DEV)
        self.ws = ((torch.rand(E, N, generator=g) + 0.5) * K ** -0.5 / 5500).to(DEV)
        mk = lambda *s: torch.empty(*s).normal_(0, 0.5, generator=g).to(TD[dtype]).to(DEV)
        self.bias = mk(E, N) if bias else None
        q = 16 // TD[dtype].itemsize
        ldy = (self.oc + q - 1) // q * q + gap * q
        self.res = mk(rows, ldy)[:, :self.oc] if residual else None
        self.yb = torch.full((rows, ldy), float("nan"), dtype=TD[dtype], device=DEV)
        self.y = self.yb[:, :self.oc]
        self.m = ds4.make_matmul_int8(K, N, groups=E, dtype=dtype, act=act, ldx=ldx, ldw=ldw, ldy=ldy)

    def workspace(self):
        n = ds4.matmul_int8_workspace_bytes(self.m, self.rows)
        return torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) if n else None

    def run(self, y=None, ws="own", stream=None, residual=None):
        y = self.y if y is None else y
        ws = self.workspace() if isinstance(ws, str) else ws
        if self.off is None:
            ds4.linear_int8(self.m, self.rows, self.x, self.xs, self.w, self.ws, y, bias=self.bias,
                            residual=self.res if residual is None else residual, workspace=ws, stream=stream)
        else:
            ds4.grouped_matmul_int8(self.m, self.rows, self.x, self.xs, self.w, self.ws, self.off, y,
                                    sorted_pair=self.pairs, top_k=max(self.k, 1), x_rows=self.x_rows, bias=self.bias,
                                    workspace=ws, stream=stream)
        return y

    def check(self, y=None):
        y = self.y if y is None else y
        for e, (a, b) in enumerate(zip(self.off_h[:-1], self.off_h[1:])):
            if a == b:
                continue
            at = self.src[a:b]
            s = torch.matmul(self.x[at].double(), self.w[e].double().t())      # (exact: below 2^53)
            z = s * self.xs[at].double()[:, None] * self.ws[e].double()
            size = z.abs()
            if self.bias is not None:
                z = z + self.bias[e].double()
                size = size + self.bias[e].double().abs()
            dz = 4 * EPS * size
            v = act64(z, self.act)
            if self.act == "swiglu":
                g, u = z.chunk(2, 1)
                dg, du = dz.chunk(2, 1)
                sg = (g * torch.sigmoid(g)).abs()
                tol = (1.13 * dg + 16 * EPS * sg) * u.abs() + sg * du + EPS * v.abs()
                tol = tol + (1.13 * dg) * du
            elif self.act in ("none", "relu"):
                tol = dz
            else:
                tol = 1.13 * dz + 16 * EPS * v.abs() + 16 * EPS * z.abs()
            if self.res is not None:
                v = v + self.res[a:b].double()
                tol = tol + EPS * (v.abs() + tol)
            tol = tol + HALF[self.dtype] * (v.abs() + tol) + 1e-37
            bad = (y[a:b].double() - v).abs() > tol
            assert not bad.any(), (e, bad.nonzero()[:4].tolist(), float(((y[a:b].double() - v).abs() / tol).max()))
        assert y[self.off_h[-1]:].isnan().all() and y[:self.off_h[0]].isnan().all()
        assert self.yb[:, self.oc:].isnan().all()


DENSE = [(1, 1, 1), (1, 7168, 7168), (2, 15, 3), (5, 33, 70), (8, 256, 512), (9, 300, 129), (16, 2048, 1000),
         (17, 100, 64), (31, 1031, 65), (64, 8192, 512), (65, 128, 257), (130, 511, 130), (300, 1000, 513),
         (257, 2047, 1030), (1000, 640, 2050)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,N", DENSE)
def test_linear_sizes(rows, K, N, dtype):
    for gap in (0, 1):
        p = Problem(rows, K, N, dtype, bias=gap == 1, residual=gap == 0, gap=gap, seed=rows + K)
        p.run()
        p.check()


@pytest.mark.parametrize("rows", [1, 7, 40, 150])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_linear_acts(act, dtype, rows):
    for N in (130, 516):
        p = Problem(rows, 300, N, dtype, act=act, bias=True, residual=True, seed=rows)
        p.run()
        p.check()


@pytest.mark.parametrize("rows,K,N,act", [(4096, 500, 4100, "swiglu"), (2045, 2050, 7170, "none"), (1021, 7170, 1026, "gelu"),
                                          (4090, 1162, 2042, "none"), (700, 5000, 1026, "swiglu"), (16, 7168, 40000, "none"),
                                          (300, 7168, 100, "silu"), (24, 8192, 2048, "swiglu"), (2048, 3000, 1024, "none")])
def test_larger_shapes(rows, K, N, act):
    """The wide tiles, splits of the contraction, a wide head."""
    p = Problem(rows, K, N, "bf16", act=act, bias=True, seed=rows)
    p.run()
    p.check()


GROUPS = [[3], [0, 5, 0], [16, 17, 1, 15, 0, 33], [1] * 40, [200, 0, 129, 64, 65], [0, 0, 700, 1], [2, 300] * 6,
          [9] * 100 + [0] * 155 + [70]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("groups", GROUPS, ids=lambda g: "-".join(map(str, g))[:30])
def test_grouped(groups, dtype):
    for k, act, N, extra in ((0, "none", 200, 0), (3, "swiglu", 130, 0), (2, "gelu", 67, 7)):
        p = Problem(sum(groups) + extra, 259, N, dtype, act=act, groups=groups, gather_k=k, bias=k > 0, gap=k % 2,
                    seed=k)
        p.run()
        p.check()


@pytest.mark.parametrize("groups", [[2600, 0, 1, 3000, 900, 1100, 30, 369], [1] * 3 + [0, 700, 150, 260, 5] * 3 + [90] * 7,
                                    [40] * 64])
def test_large_grouped_shapes(groups):
    for K, N, k, act in ((2048, 1030, 0, "none"), (1000, 2060, 4, "swiglu"), (4000, 300, 2, "none")):
        p = Problem(sum(groups), K, N, "bf16", act=act, groups=groups, gather_k=k, seed=k)
        p.run()
        p.check()


@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("K", [256, 520, 1031, 4100])
def test_few_rows(rows, K):
    for act, N in (("none", 1003), ("swiglu", 1006)):
        p = Problem(rows, K, N, "bf16", act=act, bias=True, residual=True, seed=K)
        p.run()
        p.check()


def test_largest_sums():
    """The longest contraction of the most negative code: the largest sum that 31 bits have to hold."""
    K = 131071
    for rows in (1, 40):
        x = torch.full((rows, 131072), -128, dtype=torch.int8, device=DEV)
        w = torch.full((48, 131072), -128, dtype=torch.int8, device=DEV)
        w[1::2] = 127
        y = torch.empty(rows, 48, device=DEV)
        m = ds4.make_matmul_int8(K, 48, dtype="f32", ldx=131072, ldw=131072)
        n = ds4.matmul_int8_workspace_bytes(m, rows)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
        ds4.linear_int8(m, rows, x[:, :K], torch.ones(rows, device=DEV), w[:, :K], torch.ones(48, device=DEV), y, workspace=ws)
        assert (y[:, 0::2] == float(128 * 128 * K)).all()      # (2^31 - 2^14: a multiple of 2^7, exact in fp32)
        want = torch.tensor(-128.0 * 127 * K, dtype=torch.float64).float().item()
        assert (y[:, 1::2] == want).all()


def test_nan_scale_stays_in_its_row():
    p = Problem(40, 200, 96, "f32", groups=[20, 20], gather_k=2, seed=3)
    p.xs[7] = float("nan")
    p.run()
    assert torch.equal(p.y.isnan().any(1), p.src == 7) and torch.equal(p.y.isnan().all(1), p.src == 7)


def test_residual_in_place_and_determinism():
    for rows in (3, 200):
        p = Problem(rows, 2000, 512, "bf16", act="gelu", bias=True, residual=True, seed=rows)
        p.run()
        y = p.res.clone()
        p.run(y=y, residual=y)
        assert torch.equal(y, p.y)


def test_corrupt_offsets_and_pairs_stay_inside():
    p = Problem(100, 128, 64, "f32", groups=[50, 50], gather_k=2, seed=4)
    p.pairs[::3] = -7
    p.pairs[1::3] = 2 ** 30
    p.off[1] = 1000
    p.run()
    q = Problem(12, 128, 64, "f32", groups=[6, 6], gather_k=2, seed=4)
    q.off[1] = -5
    q.pairs[0] = -1
    q.run()
    torch.cuda.synchronize()


@pytest.mark.parametrize("which", ["weights", "rows"])
def test_far_rows(which):
    """Codes more than 2^32 bytes into their tensor."""
    g = torch.Generator().manual_seed(6)
    if which == "weights":
        E, N, K, rows = 70, 8192, 8192, 6
        w = torch.zeros(E, N, K, dtype=torch.int8, device=DEV)
        some = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8).to(DEV)
        w[E - 1] = some
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[E] = rows
        for r in (rows, 200):
            off[E] = r
            x = torch.randint(-128, 128, (r, K), generator=g, dtype=torch.int8).to(DEV)
            m = ds4.make_matmul_int8(K, N, groups=E, dtype="f32")
            ws = torch.empty(ds4.matmul_int8_workspace_bytes(m, 200), dtype=torch.uint8, device=DEV)
            y = torch.empty(r, N, device=DEV)
            one = torch.ones(E, N, device=DEV)
            ds4.grouped_matmul_int8(m, r, x, torch.ones(r, device=DEV), w, one, off.to(DEV), y, workspace=ws)
            want = torch.matmul(x.double(), some.double().t())
            assert ((y.double() - want).abs() <= EPS * want.abs()).all()
    else:
        K, x_rows = 8192, (1 << 19) + 30
        x = torch.zeros(x_rows, K, dtype=torch.int8, device=DEV)
        at = torch.tensor([x_rows - 1, 5, x_rows - 30, 1 << 19, 0, 77], dtype=torch.int32, device=DEV)
        x[at.long()] = torch.randint(-128, 128, (6, K), generator=g, dtype=torch.int8).to(DEV)
        w = torch.randint(-128, 128, (1, 96, K), generator=g, dtype=torch.int8).to(DEV)
        m = ds4.make_matmul_int8(K, 96, dtype="f32")
        for rep in (1, 6):
            pairs = at.repeat(rep * rep)
            n = pairs.numel()
            wsb = ds4.matmul_int8_workspace_bytes(m, n)
            y = torch.empty(n, 96, device=DEV)
            ds4.grouped_matmul_int8(m, n, x, torch.ones(x_rows, device=DEV), w, torch.ones(1, 96, device=DEV),
                                    torch.tensor([0, n], dtype=torch.int32, device=DEV), y, sorted_pair=pairs, top_k=1,
                                    x_rows=x_rows, workspace=torch.empty(max(wsb, 16), dtype=torch.uint8, device=DEV))
            want = torch.matmul(x[pairs.long()].double(), w[0].double().t())
            assert ((y.double() - want).abs() <= EPS * want.abs()).all()


@pytest.mark.parametrize("kw", [dict(rows=4, K=700, N=300), dict(rows=64, K=8192, N=512),
                                dict(rows=200, K=300, N=600, groups=[50, 0, 149, 1], gather_k=2)])
def test_graph_replays_and_streams(kw):
    p = Problem(**kw, seed=1)
    want = p.run().clone()
    a, b = torch.empty_like(p.yb)[:, :p.oc], torch.empty_like(p.yb)[:, :p.oc]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    w1, w2 = p.workspace(), p.workspace()
    torch.cuda.synchronize()
    for _ in range(3):
        p.run(y=a, ws=w1, stream=s1)
        p.run(y=b, ws=w2, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(y=a, ws=w1)
        p.run(y=b, ws=w1)        # (one after the other: they may share a workspace)
    for i in range(3):
        p.x.copy_(torch.roll(p.x, 1, 0))
        p.xs.mul_(1.25)
        want = p.run().clone()
        a.zero_()
        b.zero_()
        w1.fill_(0x5A) if w1 is not None else None
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want)


@pytest.mark.parametrize("rows,K,N,act", [(1500, 64, 72, "none"), (900, 300, 130, "swiglu"), (9000, 200, 64, "silu"),
                                          (40, 2000, 33, "none")])
def test_1024_groups(rows, K, N, act):
    """The most groups, most of them empty or of one row: by the few-row kernel, by tiles that scan, by a plan."""
    g = torch.Generator().manual_seed(rows)
    groups = torch.bincount(torch.randint(0, 1024, (rows,), generator=g), minlength=1024).tolist()
    for k in (0, 5):
        p = Problem(rows, K, N, "bf16", act=act, groups=groups, gather_k=k, bias=True, seed=k)
        p.run()
        p.check()


@pytest.mark.parametrize("groups", [[40], [300], [700, 5], [3, 0, 9]])
def test_offsets_that_start_behind_zero(groups):
    """Rows before the first group and behind the last are left as they were."""
    first, behind = 7, 11
    n = sum(groups)
    p = Problem(first + n + behind, 330, 150, "f32", groups=groups, bias=True, seed=n)
    p.off += first
    p.off_h = [o + first for o in p.off_h]
    p.run()
    p.check()


def test_many_rows_of_one_column():
    """A product whose chunks of 16 rows are more than a grid's second dimension holds."""
    P, K = (1 << 20) + 5, 48
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-128, 128, (P, K), generator=g, dtype=torch.int8).to(DEV)
    w = torch.randint(-128, 128, (3, K), generator=g, dtype=torch.int8).to(DEV)
    y = torch.full((P, 4), float("nan"), device=DEV)
    m = ds4.make_matmul_int8(K, 3, dtype="f32", ldy=4)
    n = ds4.matmul_int8_workspace_bytes(m, P)
    ds4.linear_int8(m, P, x, torch.ones(P, device=DEV), w, torch.ones(3, device=DEV), y,
                    workspace=torch.empty(n, dtype=torch.uint8, device=DEV) if n else None)
    assert torch.equal(y[:, :3].double(), torch.matmul(x.double(), w.double().t())) and y[:, 3].isnan().all()


def test_experts_in_8_bits_to_the_next_token():
    """A layer's way through the calls: route, permute, rows to codes, gate/up products by expert, codes again, down
    products, the rows collected, the head's product, rules on its logits, sampling.  Each stage is checked against
    fp64 on the stage's own inputs."""
    T, E, k, H, F, V = 37, 16, 4, 512, 256, 3001
    g = torch.Generator().manual_seed(14)
    cfg = ds4.make_config(H, F, E, k)
    P = T * k
    x = torch.empty(T, H).normal_(generator=g).bfloat16().to(DEV)
    logits = torch.empty(T, E).normal_(generator=g).to(DEV)

    def weights(n, K):
        w = torch.empty(n, K).normal_(0, K ** -0.5, generator=g).to(DEV)
        c, s = torch.empty(n, K, dtype=torch.int8, device=DEV), torch.empty(n, device=DEV)
        ds4.quantize_rows_int8(n, K, w, c, s)
        return c, s

    w1, s1 = weights(E * 2 * F, H)
    w2, s2 = weights(E * H, F)
    wh, sh = weights(V, H)
    idx, tw = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    off, sp, pp, act = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (E + 1, P, P, E + 1))
    ds4.route(cfg, T, logits, idx, tw)
    ds4.permute(cfg, T, idx, off, sp, pp, act)
    m1 = ds4.make_matmul_int8(H, 2 * F, groups=E, act="swiglu")
    m2 = ds4.make_matmul_int8(F, H, groups=E)
    mh = ds4.make_matmul_int8(H, V, dtype="f32", ldy=3004)
    ws = torch.empty(max(ds4.matmul_int8_workspace_bytes(m, r) for m, r in ((m1, P), (m2, P), (mh, T))), dtype=torch.uint8,
                     device=DEV)

    def quantized(t):
        c, s = torch.empty(t.shape, dtype=torch.int8, device=DEV), torch.empty(t.shape[0], device=DEV)
        ds4.quantize_rows_int8(*t.shape, t, c, s)
        return c, s

    xc, xs = quantized(x)
    h = torch.empty(P, F, dtype=torch.bfloat16, device=DEV)
    ds4.grouped_matmul_int8(m1, P, xc, xs, w1, s1, off, h, sorted_pair=sp, top_k=k, x_rows=T, workspace=ws)
    hc, hs = quantized(h)
    eo, y = torch.empty(P, H, dtype=torch.bfloat16, device=DEV), torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    ds4.grouped_matmul_int8(m2, P, hc, hs, w2, s2, off, eo, workspace=ws)
    ds4.collect(ds4.make_rows(H, k), T, P, eo, pp, y, topk_w=tw, base=x)
    yc, ys = quantized(y)
    out = torch.empty(T, 3004, device=DEV)
    ds4.linear_int8(mh, T, yc, ys, wh, sh, out, workspace=ws)
    lg = out[:, :V]
    mask = torch.full((1, (V + 31) // 32), 0x55555555, dtype=torch.int32, device=DEV)
    ds4.adjust_logits(T, V, lg, lg, bias_token=torch.zeros(1, dtype=torch.int32, device=DEV),
                      bias_value=torch.full((1,), float("-inf"), device=DEV),
                      bias_offsets=torch.cat([torch.zeros(1), torch.ones(T)]).int().to(DEV), mask=mask,
                      mask_row=torch.zeros(T, dtype=torch.int32, device=DEV))
    token = torch.empty(T, dtype=torch.int32, device=DEV)
    sws = torch.empty(max(1, ds4.sample_workspace_bytes(T, V)), dtype=torch.uint8, device=DEV)
    ds4.sample(T, V, lg, torch.zeros(T, device=DEV), token, temperature=torch.zeros(T, device=DEV), workspace=sws)

    # (sums of codes first, which fp64 holds exactly: a sum of 0 is 0 on both sides)
    def near(got, want, sums):
        """Half a step of bf16 and the roundings of the fp32 epilogue, 32 of them at most."""
        assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 32 * EPS * sums).all()

    ex = torch.repeat_interleave(torch.arange(E, device=DEV), (off[1:] - off[:-1]).long())
    src = (sp // k).long()
    z = torch.matmul(w1.double().view(E, 2 * F, H)[ex], xc.double()[src][:, :, None])[:, :, 0]
    z = z * xs.double()[src][:, None] * s1.double().view(E, 2 * F)[ex]
    gt, up = z.chunk(2, 1)
    near(h, gt * torch.sigmoid(gt) * up, gt.abs() * up.abs())
    e = torch.matmul(w2.double().view(E, H, F)[ex], hc.double()[:, :, None])[:, :, 0]
    e = e * hs.double()[:, None] * s2.double().view(E, H)[ex]
    near(eo, e, e.abs())
    pairs = eo.double()[pp.long()].view(T, k, H) * tw.double()[:, :, None]
    near(y, x.double() + pairs.sum(1), x.double().abs() + pairs.abs().sum(1))
    want = torch.matmul(yc.double(), wh.double().t()) * ys.double()[:, None] * sh.double()
    allowed = (torch.arange(V, device=DEV) % 2 == 0)[None].expand(T, V).clone()
    allowed[0, 0] = False
    assert ((lg.double() - want).abs()[allowed] <= 4 * EPS * want.abs()[allowed]).all()
    assert (lg[~allowed] == float("-inf")).all()
    assert torch.equal(token.long(), torch.where(allowed, lg, float("-inf")).argmax(1))


# rows, K, N, groups (None: dense): the wide tiles of 128 rows with and without their pipeline, and contractions
# in 2, 4, 8 and 16 parts, whose ends leave a part with fewer steps, or rows of a tile without a row
PARTS = [(32679, 2707, 230, None), (69, 11360, 9010, None), (4165, 10355, 82, None), (2055, 16263, 126, None),
         (59, 15945, 286, None), (53, 2762, 4826, None), (3485, 3391, 62, None), (19, 15416, 2122, None),
         (736, 2157, 494, [2] * 128 + [0] * 64 + [1] * 32 + [14] * 32),
         (24, 3806, 10590, [0, 17, 1, 1, 0, 3, 1, 1]), (120, 5625, 1402, [100, 0, 3, 1, 0, 16, 0, 0]),
         (616, 12114, 118, [0, 129, 64, 1, 0, 300, 65, 57]), (1351, 15895, 54, [1000, 0, 55, 296]),
         (2195, 6312, 62, [34] * 64 + [0]), (4446, 10690, 66, [4000, 1, 0, 128, 129, 60, 64, 64]),
         (2733, 1197, 5814, None)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,N,groups", PARTS, ids=lambda v: str(v)[:12])
def test_wide_tiles_and_parts(rows, K, N, groups, dtype):
    for act, k in (("none", 0), ("swiglu", 3)):
        rows_ = rows if groups is None else sum(groups)
        p = Problem(rows_ + (5 if groups else 0), K, N, dtype, act=act, groups=groups, gather_k=k if groups else 0,
                    bias=True, residual=groups is None, gap=1, seed=k)
        first = p.run()[:rows_].clone()
        p.check()
        assert torch.equal(p.run()[:rows_], first)


@pytest.mark.parametrize("rows,K,N,groups", [(69, 11360, 9010, None), (59, 15945, 286, None), (53, 2762, 4826, None),
                                             (120, 5625, 1402, [100, 0, 3, 1, 0, 16, 0, 0])], ids=lambda v: str(v)[:12])
def test_parts_in_a_graph(rows, K, N, groups):
    """The sums of the parts are written anew on every replay, whatever the workspace holds by then."""
    p = Problem(rows, K, N, "bf16", act="silu", groups=groups, bias=True)
    want = p.run().clone()
    p.check()
    ws, y = p.workspace(), torch.empty_like(p.yb)[:, :p.oc]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(y=y, ws=ws)
    for _ in range(3):
        y.zero_()
        ws.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert torch.equal(p.run(), want)
