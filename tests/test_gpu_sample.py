"""ds4moe_sample against the definition evaluated on the host in fp64.

Tokens must be equal: a running sum would have to come within 2^-40 of a border
for the kernel's 2^-43 weights to choose another token than fp64 does, which
the random cases do not (asserted in the reference).  Probabilities are one
fp32 rounding (2^-24) of a quotient whose terms are off by at most V * 2^-43 in
all."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402

INF = float("inf")


def reference(l, T, k, p, q, u, margin=2.0 ** -40):
    """(token, prob) of one row of fp64 logits (numpy)."""
    idx = np.nonzero(l > -INF)[0]        # (NaN compares false)
    if idx.size == 0:
        return -1, 0.0
    order = idx[np.argsort(-l[idx], kind="stable")]
    if not T > 0:
        return int(order[0]), 1.0
    v = l[order]
    d = np.where(v == v[0], 0.0, v[0] - v) / T
    w = np.exp(-d)
    if k > 0:
        w = w[:k]
    if p < 1:
        c = np.cumsum(w)
        t = p * c[-1]
        n = int(np.argmax(c >= t)) + 1
        assert p <= 0 or np.abs(c - t).min() > margin * c[-1] or n == 1, "top-p border"
        w = w[:n]
    if q > 0:
        assert np.abs(w[1:] - q).min(initial=1) > margin or q >= 1, "min-p border"
        w = w[: max(1, int((w >= q).sum()))]
    c = np.cumsum(w)
    t = min(max(u, 0.0), 1.0) * c[-1]
    i = min(int((c <= t).sum()), len(w) - 1) if u < 1 else int(np.nonzero(w > 2.0 ** -44)[0][-1])
    assert not 0 < u < 1 or np.abs(c - t).min() > margin * c[-1], "border of u"
    return int(order[i]), float(w[i] / c[-1])


def check(logits, T=None, k=None, p=None, q=None, u=None, seed=0):
    """Runs rows of `logits` (any dtype, on the host) and compares every row."""
    B, V = logits.shape
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(B, generator=g) if u is None else torch.as_tensor(u, dtype=torch.float32).expand(B).contiguous()
    par = []
    for x, dt in ((T, torch.float32), (k, torch.int32), (p, torch.float32), (q, torch.float32)):
        par.append(None if x is None else torch.as_tensor(x, dtype=dt).expand(B).contiguous())
    dev = [None if x is None else x.to(DEV) for x in par]
    token = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    prob = torch.full((B,), float("nan"), device=DEV)
    n = ds4.sample_workspace_bytes(B, V)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) if n else None
    lg = logits.to(DEV) if logits.is_contiguous() else torch.empty_strided(
        logits.shape, logits.stride(), dtype=logits.dtype, device=DEV).copy_(logits)
    ds4.sample(B, V, lg, u.to(DEV), token, *dev, prob=prob, workspace=ws)
    tok, pr = token.cpu().tolist(), prob.cpu().double().tolist()
    host = logits.double().numpy()
    get = lambda x, r, d: d if x is None else float(x[r])
    for r in range(B):
        T_, k_, p_, q_ = (get(x, r, d) for x, d in zip(par, (1.0, 0, 2.0, 0.0)))
        want, wp = reference(host[r], T_, int(k_), p_, q_, float(u[r]))
        assert tok[r] == want, (r, tok[r], want, T_, k_, p_, q_, float(u[r]))
        assert abs(pr[r] - wp) <= 2.0 ** -24 * wp + V * 2.0 ** -43, (r, pr[r], wp)
    return token


def normal(B, V, std=2.0, seed=1, dtype=torch.float32):
    return torch.empty(B, V).normal_(0, std, generator=torch.Generator().manual_seed(seed)).to(dtype)


SIZES = [1, 2, 3, 17, 63, 64, 65, 1000, 1023, 1025, 4096, 4097, 16385, 32003, 50003, 131072]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_sizes_and_filters(V, dtype):
    print(f"sample V={V} {dtype}", flush=True)
    B = 9
    l = normal(B, V, 2.0, V, dtype)
    check(l, seed=1)
    check(l, T=0.7, seed=2)
    check(l, k=max(1, V // 3), seed=3)
    check(l, p=0.83, seed=4)
    check(l, q=0.0371, seed=5)
    check(l, T=1.3, k=40, p=0.9, q=0.011, seed=6)
    check(l, T=torch.tensor([0.0, 1.0, 0.2, 3.0, -1.0, 0.5, 1.0, 2.0, 0.01]), k=torch.arange(9),
          p=torch.tensor([0.5, 0.1, 1.0, 0.99, 0.2, 0.0, 0.7, 1.5, 0.6]),
          q=torch.tensor([0.0, 0.5, 0.1, 0.003, 0.0, 1.0, 2.0, 0.001, 0.0]), seed=7)


@pytest.mark.parametrize("B,V", [(1, 131072), (64, 32000), (300, 1001)])
def test_batches(B, V):
    g = torch.Generator().manual_seed(B)
    check(normal(B, V, 3.0, B), T=0.2 + torch.rand(B, generator=g), k=torch.randint(0, 300, (B,), generator=g),
          p=0.3 + 0.8 * torch.rand(B, generator=g), q=0.05 * torch.rand(B, generator=g))


def test_flat_rows_cross_deep_in_the_order():
    """Many tokens of like weight: borders in crowded bins, found by narrowing their range."""
    l = normal(6, 60000, 0.004, 5)
    check(l, seed=1)
    check(l, p=0.6, seed=2)
    check(l, k=30001, seed=3)
    check(l, T=2.0, k=50000, p=0.97, q=0.9951, seed=4)
    check(normal(4, 131072, 0.1, 6), T=5.0, p=0.5, seed=5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_ties_go_to_the_lowest_index(dtype):
    V = 20001
    g = torch.Generator().manual_seed(3)
    for l in (torch.zeros(4, V), torch.randint(0, 2, (4, V), generator=g).float(),
              torch.randint(-3, 1, (4, V), generator=g).float() * 0.01, torch.full((4, V), -0.0)):
        l = l.to(dtype)
        check(l, u=torch.tensor([0.0, 0.25001, 0.70003, 0.99999]))
        check(l, k=777, u=torch.tensor([0.0, 0.2503, 0.7001, 0.999]))
        check(l, k=1, u=0.9)
        check(l, p=0.31234, u=torch.tensor([0.0, 0.25003, 0.70013, 0.9999]))
        check(l, T=0.0)


def test_masks():
    """Masked tokens (-infinity, NaN, the type's lowest value) and rows with nothing left."""
    V = 3000
    l = normal(8, V)
    l[0] = -INF
    l[1] = float("nan")
    l[2, 1:] = -INF
    l[3, :-1] = float("nan")
    l[4, ::2] = -INF
    l[5, 5:] = torch.finfo(torch.float32).min
    l[6, [7, 1234, 2999]] = INF
    l[7] = torch.finfo(torch.float32).min
    for kw in ({}, dict(k=10), dict(p=0.8), dict(q=0.02), dict(T=0.0), dict(T=0.8, k=50, p=0.9, q=0.01)):
        check(l, **kw)
    check(l.to(torch.bfloat16)[[0, 1, 2, 3, 4, 6]], k=20, p=0.9)


def test_extreme_parameters():
    l = normal(5, 5000)
    check(l, T=1e-30)
    check(l, T=torch.tensor([1e-44, 1e-10, 1e4, 1e30, INF]))
    check(l, T=float("nan"))
    check(l, k=torch.tensor([-5, 2 ** 31 - 1, 5000, 4999, 1]))
    check(l, p=torch.tensor([-1.0, 0.0, 1e-30, 1.0, INF]))
    check(l, q=torch.tensor([-1.0, 1e-30, 1.0, INF, 0.5]))
    check(l, u=0.0)
    check(l, u=torch.tensor([-3.0, 0.0, 2.0 ** -24, 1 - 2.0 ** -24, 2.0 ** -60]))
    check(l * 100)
    check(normal(3, 5000) * 1e30)


def test_u_outside_counts_as_nearest():
    l = normal(3, 100)
    check(l, k=7, u=torch.tensor([1.0, 1.5, INF]))
    check(l, k=7, u=torch.tensor([-1.0, -INF, 0.0]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_strided_rows(dtype):
    """Rows at any distance and alignment; what lies between them is not read as a logit."""
    for ld in (1003, 1024, 1500):
        t = torch.full((7, ld), 1e4, dtype=dtype)
        t[:, :1003] = normal(7, 1003, 2.0, ld, dtype)
        check(t[:, :1003], k=30, p=0.9)


def test_head_and_sample_as_used():
    """The output head's products feeding the sampler, greedy and sampled, on a batch of sessions."""
    B, H, V = 5, 512, 6001
    g = torch.Generator().manual_seed(9)
    x = torch.empty(B, H).normal_(generator=g).to(torch.bfloat16).to(DEV)
    w = torch.empty(V, H).normal_(0, 0.1, generator=g).to(torch.bfloat16).to(DEV)
    ld = (V + 7) // 8 * 8
    logits = torch.zeros(B, ld, dtype=torch.bfloat16, device=DEV)
    m = ds4.make_matmul(H, V, ldy=ld)
    ds4.linear(m, B, x, w, logits)
    view = logits[:, :V]
    exact = x.double() @ w.double().t()
    assert ((view.double() - exact).abs() <= 2.0 ** -8 * exact.abs() + 1e-3).all()
    u = torch.rand(B, generator=g).to(DEV)
    token = torch.empty(B, dtype=torch.int32, device=DEV)
    T = torch.tensor([0.0, 1.0, 0.7, 0.0, 1.2])
    k = torch.tensor([0, 50, 0, 0, 9], dtype=torch.int32)
    ws = torch.empty(ds4.sample_workspace_bytes(B, V), dtype=torch.uint8, device=DEV)
    ds4.sample(B, V, view, u, token, temperature=T.to(DEV), top_k=k.to(DEV), workspace=ws)
    host = view.double().cpu().numpy()
    for r in range(B):
        assert int(token[r]) == reference(host[r], float(T[r]), int(k[r]), 2.0, 0.0, float(u[r]))[0]


def test_distribution_of_many_draws():
    """Evenly spaced u give every token its probability to within one part in the number of draws."""
    n = 4000
    l = normal(1, 50, 1.5, 8).expand(n, 50).contiguous()
    u = (torch.arange(n) + 0.5) / n
    tok = check(l, T=0.9, k=20, u=u)
    counts = torch.bincount(tok.cpu().long(), minlength=50).double() / n
    w = torch.softmax(torch.topk(l[0].double() / float(np.float32(0.9)), 20).values, 0)
    want = torch.zeros(50, dtype=torch.float64)
    want[torch.topk(l[0], 20).indices] = w
    assert (counts - want).abs().max() <= 1.0 / n + 1e-9


def test_graph_replays():
    B, V = 3, 32003
    ls = [normal(B, V, 2.0, s).to(DEV) for s in range(3)]
    u = torch.rand(B, generator=torch.Generator().manual_seed(2)).to(DEV)
    kw = dict(temperature=torch.full((B,), 0.8, device=DEV), top_k=torch.full((B,), 60, dtype=torch.int32, device=DEV),
              top_p=torch.full((B,), 0.95, device=DEV))
    n = ds4.sample_workspace_bytes(B, V)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    l, token, prob = ls[0].clone(), torch.empty(B, dtype=torch.int32, device=DEV), torch.empty(B, device=DEV)
    call = lambda: ds4.sample(B, V, l, u, token, prob=prob, workspace=ws, **kw)
    refs = []
    for x in ls:
        l.copy_(x)
        call()
        refs.append((token.clone(), prob.clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call()
    for rep in range(6):
        l.copy_(ls[rep % 3])
        token.fill_(-9)
        torch.randn(1000, device=DEV).sum().item()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(token, refs[rep % 3][0]) and torch.equal(prob, refs[rep % 3][1]), rep


def test_crowded_bin_beside_an_outlier():
    """A far low logit keeps the bins wide, so that nearly all tokens share one and its range is narrowed."""
    l = normal(5, 60000, 0.004, 15)
    l[:, 777] = -50.0
    check(l, seed=1)
    check(l, p=0.6, seed=2)
    check(l, k=30001, seed=3)
    check(l, T=2.0, k=50000, p=0.97, q=0.9951, seed=4)
    short = l[:, :9000].contiguous()
    check(short, k=5001, p=0.8, seed=5)
    check(short.to(torch.bfloat16), p=0.7, seed=6)
