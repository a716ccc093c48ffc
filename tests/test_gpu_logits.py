"""Rules on logits (ds4moe_adjust_logits) against their definition in fp64, row
by row.

Bounds: a token that no rule names is copied exactly (rounded once where the
output is bf16 and the input fp32).  Otherwise at most six fp32 operations
(division or product, frequency * n, two subtractions, the bias's addition),
each within 2^-24 of the values it takes, whose sizes are at most |l'| +
|frequency n| + |presence| + |bias|, and the output's rounding (bf16 2^-8, fp32
2^-24 of the value).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
INF = float("inf")


class Case:
    def __init__(self, B, V, dtype="f32", out="f32", history=50, bias=5, mask="some", penalties="rpf", prompt=True,
                 gap=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.V, self.out_t = B, V, out
        buf = torch.full((B, V + gap), float("nan"), dtype=TD[dtype])
        buf[:, :V] = torch.empty(B, V).normal_(0, 3, generator=g)
        buf[:, :V][torch.rand(B, V, generator=g) < 0.05] = -INF
        self.logits_h = buf[:, :V].clone()
        self.logits = buf.to(DEV)[:, :V]
        self.kw, self.h = {}, {}

        def add(name, t):
            self.h[name] = t
            self.kw[name] = t.to(DEV)

        def ragged(most):
            n = torch.randint(0, most + 1, (B,), generator=g)
            n[torch.randint(0, B, (1,), generator=g)] = most
            if B > 2:
                n[1] = 0
            off = torch.zeros(B + 1, dtype=torch.int32)
            off[1:] = n.cumsum(0)
            return off

        if history:
            off = ragged(history)
            n = int(off[-1])
            tok = (V * torch.rand(n, generator=g).pow(3)).int().clamp(max=V - 1)
            tok[torch.rand(n, generator=g) < 0.05] = -1                # padding
            tok[torch.rand(n, generator=g) < 0.02] = V + 3
            add("history", tok)
            add("history_offsets", off)
            if prompt:
                add("prompt_len", torch.randint(-2, history + 3, (B,), generator=g).int())
            if "r" in penalties:
                add("repetition", 0.6 + torch.rand(B, generator=g))
            if "p" in penalties:
                add("presence", torch.randn(B, generator=g))
            if "f" in penalties:
                add("frequency", torch.randn(B, generator=g))
        if bias:
            off = ragged(bias)
            n = int(off[-1])
            tok = torch.randint(-2, V + 2, (n,), generator=g).int()    # some twice, some outside
            val = 4 * torch.randn(n, generator=g)
            val[torch.rand(n, generator=g) < 0.3] = -INF
            add("bias_token", tok)
            add("bias_value", val)
            add("bias_offsets", off)
        if mask:
            W = (V + 31) // 32
            rows = B if mask == "own" else 3
            bits = torch.randint(-2 ** 31, 2 ** 31, (rows, W + gap), generator=g, dtype=torch.int64)
            bits[torch.rand(rows, W + gap, generator=g) < 0.4] = 0
            bits[0] = 0                                                # leaves nothing
            self.h["mask"] = bits.int()
            self.kw["mask"] = bits.int().to(DEV)[:, :W]
            if mask != "own":
                add("mask_row", torch.randint(-1, rows + 1, (B,), generator=g).int())
        self.out_buf = torch.full((B, V + 2 * gap), float("nan"), dtype=TD[out], device=DEV)
        self.out = self.out_buf[:, :V]

    def run(self, out=None, logits=None, **kw):
        out = self.out if out is None else out
        ds4.adjust_logits(self.B, self.V, self.logits if logits is None else logits, out, **self.kw, **kw)
        return out

    def want(self):
        """Values and sizes (what the bounds count) in fp64."""
        h, V = self.h, self.V
        val, size = self.logits_h.double(), self.logits_h.double().abs()
        touched = torch.zeros(self.B, V, dtype=torch.bool)
        for b in range(self.B):
            l, sz = val[b], size[b]
            if "history" in h:
                said = h["history"][h["history_offsets"][b]:h["history_offsets"][b + 1]].long()
                p = max(int(h["prompt_len"][b]), 0) if "prompt_len" in h else 0
                inside = (said >= 0) & (said < V)
                c = torch.bincount(said[inside], minlength=V)
                n = torch.bincount(said[p:][inside[p:]], minlength=V)
                if "repetition" in h:
                    r = h["repetition"][b].double()
                    l = torch.where(c > 0, torch.where(l > 0, l / r, l * r), l)
                    touched[b] |= c > 0
                sz = l.abs()
                f = h["frequency"][b].double() if "frequency" in h else 0.0
                q = h["presence"][b].double() if "presence" in h else 0.0
                l = torch.where(n > 0, l - f * n - q, l)
                sz = sz + (n > 0) * (abs(f) * n + abs(q))
                touched[b] |= n > 0
            if "bias_token" in h:
                for i in range(int(h["bias_offsets"][b]), int(h["bias_offsets"][b + 1])):
                    t = int(h["bias_token"][i])
                    if 0 <= t < V and not any(int(x) == t for x in h["bias_token"][i + 1:h["bias_offsets"][b + 1]]):
                        l[t] += h["bias_value"][i].double()
                        sz[t] += h["bias_value"][i].double().abs()
                        touched[b, t] = True
            if "mask" in h:
                g = int(h["mask_row"][b]) if "mask_row" in h else b
                if 0 <= g < h["mask"].shape[0]:
                    words = h["mask"][g].long() & 0xFFFFFFFF
                    bit = (words[:, None] >> torch.arange(32)) & 1
                    l = torch.where(bit.reshape(-1)[:V] == 1, l, torch.full((), -INF, dtype=torch.float64))
            val[b], size[b] = l, sz
        return val, size, touched

    def check(self, out=None):
        out = self.out if out is None else out
        got = out.cpu().double()
        val, size, touched = self.want()
        fin = torch.isfinite(val)
        assert torch.equal(got[~fin], val[~fin])
        tol = torch.where(touched, 6 * 2.0 ** -24 * size, torch.zeros_like(size)) + HALF[self.out_t] * val.abs()
        assert ((got - val).abs()[fin] <= tol[fin]).all()
        same = fin & ~touched
        exact = self.logits_h.to(TD[self.out_t]).double()
        assert torch.equal(got[same], exact[same])
        assert self.out_buf[:, self.V:].isnan().all()


SIZES = [(1, 1), (1, 5), (2, 31), (3, 33), (7, 1000), (5, 1023), (4, 1025), (3, 4096), (9, 4099), (2, 50003), (33, 129)]


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("B,V", SIZES)
def test_all_rules(B, V, dtype, out):
    c = Case(B, V, dtype, out, gap=(B * V) % 4, seed=B + V)
    c.run()
    c.check()


@pytest.mark.parametrize("kw", [dict(history=0, bias=0, mask=None), dict(history=0, bias=0), dict(history=0, mask=None),
                                dict(bias=0, mask=None), dict(bias=0, mask=None, penalties="r"),
                                dict(bias=0, penalties="f", prompt=False), dict(bias=0, penalties="p"),
                                dict(mask="own"), dict(penalties=""), dict(history=3000, bias=400, mask="own")],
                         ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
@pytest.mark.parametrize("B,V,dtype", [(5, 2500, "f32"), (6, 2049, "bf16")])
def test_each_rule(B, V, dtype, kw):
    c = Case(B, V, dtype, seed=3, **kw)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(dtype):
    """Enough tokens in all for the larger segments, rows of odd length."""
    c = Case(130, 40007, dtype, history=300, seed=4)
    c.run()
    c.check()


def test_long_history():
    """A history of more tokens than the vocabulary, every token many times."""
    c = Case(3, 700, history=200000, bias=0, mask=None, seed=5)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place(dtype):
    c = Case(9, 3001, dtype, dtype, gap=5, seed=6)
    work = torch.full((9, 3001 + 5), float("nan"), dtype=TD[dtype], device=DEV)
    work[:, :3001] = c.logits
    c.run(out=work[:, :3001], logits=work[:, :3001])
    c.check(work[:, :3001])
    assert work[:, 3001:].isnan().all()


def test_infinities_and_nan():
    """+infinity stays, NaN stays where it is allowed, and neither shows where it is masked."""
    V = 300
    l = torch.zeros(1, V, device=DEV)
    l[0, 10:20], l[0, 20:30], l[0, 30:40] = INF, float("nan"), -INF
    bits = torch.full((1, (V + 31) // 32), -1, dtype=torch.int32)
    bits[0, 0] = ~((1 << 12) | (1 << 22))
    hist = torch.arange(8, 42, dtype=torch.int32)
    out = torch.empty(1, V, device=DEV)
    ds4.adjust_logits(1, V, l, out, history=hist.to(DEV), history_offsets=torch.tensor([0, 34], dtype=torch.int32, device=DEV),
                      repetition=torch.tensor([2.0], device=DEV), presence=torch.tensor([0.5], device=DEV),
                      mask=bits.to(DEV))
    o = out[0].cpu()
    assert o[12] == -INF and o[22] == -INF
    assert (o[[10, 11, 13, 19]] == INF).all() and o[[20, 21, 23, 29]].isnan().all() and (o[30:40] == -INF).all()
    assert o[8] == -0.5 and o[41] == -0.5 and (o[42:] == 0).all() and (o[:8] == 0).all()


def test_corrupt_offsets_are_empty_lists():
    V, B = 64, 4
    l = torch.randn(B, V, device=DEV)
    hist = torch.zeros(10, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 11, 5, -3, 10], dtype=torch.int32, device=DEV)      # every range invalid
    out = torch.empty_like(l)
    ds4.adjust_logits(B, V, l, out, history=hist, history_offsets=off, presence=torch.ones(B, device=DEV),
                      bias_token=hist, bias_value=torch.ones(10, device=DEV), bias_offsets=off)
    assert torch.equal(out, l)


def test_empty_lists():
    V, B = 100, 3
    l = torch.randn(B, V, device=DEV)
    none, off = torch.empty(0, dtype=torch.int32, device=DEV), torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    out = torch.empty_like(l)
    ds4.adjust_logits(B, V, l, out, history=none, history_offsets=off, presence=torch.ones(B, device=DEV),
                      bias_token=none, bias_value=none.float(), bias_offsets=off)
    assert torch.equal(out, l)


def test_far_rows():
    """Rows more than 2^31 elements apart in all."""
    V, ld, B = 1000, 1 << 20, 2100
    buf = torch.empty(B, ld, dtype=torch.bfloat16, device=DEV)
    vals = torch.randn(B, V, device=DEV).bfloat16()
    buf[:, :V] = vals
    out = torch.empty(B, V, device=DEV)
    ds4.adjust_logits(B, V, buf, out, bias_token=torch.tensor([7], dtype=torch.int32, device=DEV),
                      bias_value=torch.tensor([3.0], device=DEV),
                      bias_offsets=torch.cat([torch.zeros(B), torch.ones(1)]).int().to(DEV))
    want = vals.float()
    want[B - 1, 7] += 3.0
    assert torch.equal(out, want)


@pytest.mark.parametrize("B,V", [(5, 1 << 20), (32768, 9), (2, (1 << 20) - 1), (1025, 4097), (600, 8191)])
def test_limits(B, V):
    """The most tokens and rows, and borders of the segments, against torch's own scatter of one rule each."""
    g = torch.Generator().manual_seed(B)
    l = torch.empty(B, V).normal_(generator=g).to(DEV)
    n = torch.randint(0, 4, (B,), generator=g)
    off = torch.zeros(B + 1, dtype=torch.int32)
    off[1:] = n.cumsum(0)
    total = int(off[-1])
    tok = torch.randint(0, V, (total,), generator=g)
    row = torch.repeat_interleave(torch.arange(B), n)
    freq = torch.rand(B, generator=g)
    mask = torch.randint(-2 ** 31, 2 ** 31, (B, (V + 31) // 32), generator=g, dtype=torch.int64).int()
    out = torch.full((B, V), float("nan"), device=DEV)
    ds4.adjust_logits(B, V, l, out, history=tok.int().to(DEV), history_offsets=off.to(DEV), frequency=freq.to(DEV),
                      mask=mask.to(DEV))
    count = torch.zeros(B, V, dtype=torch.float64, device=DEV)
    count.index_put_((row.to(DEV), tok.to(DEV)), torch.ones(total, dtype=torch.float64, device=DEV), accumulate=True)
    want = l.double() - freq.double().to(DEV)[:, None] * count
    bit = (mask.to(DEV)[:, :, None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
    allowed = bit.reshape(B, -1)[:, :V] == 1
    assert (out[~allowed] == -INF).all()
    tol = (count > 0) * 4 * 2.0 ** -24 * (l.double().abs() + count)
    assert ((out.double() - want).abs()[allowed] <= tol[allowed]).all()


def test_then_sample():
    """Penalties, a ban and a mask carry through to the choice; a row whose mask leaves nothing has no token."""
    B, V = 6, 70001
    g = torch.Generator().manual_seed(12)
    l = torch.empty(B, V).normal_(generator=g).to(DEV)
    l[:, 500] = 20.0                                 # every row's favourite
    l[:, 60001] = 15.0
    hist = torch.full((40,), 500, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 0, 40, 40, 40, 40, 40], dtype=torch.int32, device=DEV)
    W = (V + 31) // 32
    mask = torch.zeros(2, W, dtype=torch.int32)
    mask[0, 77 // 32] = 1 << (77 % 32)
    rows = torch.tensor([-1, -1, -1, 0, 1, -1], dtype=torch.int32, device=DEV)
    ds4.adjust_logits(B, V, l, l, history=hist, history_offsets=off, frequency=torch.ones(B, device=DEV),
                      bias_token=torch.tensor([500, 60001], dtype=torch.int32, device=DEV),
                      bias_value=torch.tensor([-INF, -INF], device=DEV),
                      bias_offsets=torch.tensor([0, 0, 0, 1, 1, 1, 2], dtype=torch.int32, device=DEV),
                      mask=mask.to(DEV), mask_row=rows)
    token, prob = torch.empty(B, dtype=torch.int32, device=DEV), torch.empty(B, device=DEV)
    ws = torch.empty(ds4.sample_workspace_bytes(B, V), dtype=torch.uint8, device=DEV)
    ds4.sample(B, V, l, torch.full((B,), 0.5, device=DEV), token, top_p=torch.full((B,), 0.9, device=DEV), prob=prob,
               workspace=ws)
    t = token.tolist()
    # (20 - 40 says below every other token; the last row's only bias bans token 60001, 500 stays)
    assert t == [500, 60001, 60001, 77, -1, 500]
    assert float(prob[3]) == 1.0 and float(prob[4]) == 0.0


def test_graph_replays_and_streams():
    c = Case(20, 9001, history=500, bias=50, seed=9)
    want = torch.empty(20, 9001, device=DEV)
    c.run(out=want)
    a, b = torch.empty_like(want), torch.empty_like(want)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    c.run(out=a, stream=s1)
    c.run(out=b, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    got = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=got)
    for i in range(3):
        got.zero_()
        c.logits.mul_(1.5)
        c.kw["history"].add_(1)
        c.run(out=want)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
