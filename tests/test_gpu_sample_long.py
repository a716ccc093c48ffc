"""ds4moe_sample on rows past 16384 tokens, which several workgroups share in
four launches: masked, infinite and extreme rows, shares of a row without a
live token, padded rows, and batches of one workgroup per row.  The definition
and the tolerances are those of the short rows' tests."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402
from test_gpu_sample import INF, check, normal, reference  # noqa: E402

V = 40001
FILTERS = ({}, dict(k=10), dict(p=0.8), dict(q=0.02), dict(T=0.0), dict(T=0.8, k=50, p=0.9, q=0.01))


def masked_rows(dtype):
    """12 rows, of each of which 10 workgroups read about 4001 tokens."""
    l = normal(12, V, 2.0, 31).to(dtype)
    lowest = torch.finfo(dtype).min
    l[0] = -INF
    l[1] = float("nan")
    l[2, 1:] = -INF
    l[3, :-1] = float("nan")
    l[4, ::2] = -INF
    l[5, 5:] = lowest
    l[6, [7, 12345, 39999]] = INF
    l[7] = lowest
    l[8, :21000] = -INF          # all that lives in one share of the row
    l[8, 21040:] = float("nan")
    l[9, :30000] = -INF          # infinities in one share, live tokens in others
    l[9, 38000:38004] = INF
    l[10, 100:] = -1e4           # a mask of a large finite value
    l[11] = INF
    return l


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_masks(dtype):
    for i, kw in enumerate(FILTERS):
        print(f"masks {dtype} {kw}", flush=True)
        check(masked_rows(dtype), seed=40 + i, **kw)


def test_extreme_parameters():
    l = normal(5, V, 2.0, 32)
    for i, kw in enumerate((
            dict(T=1e-30), dict(T=torch.tensor([1e-44, 1e-10, 1e4, 1e30, INF])), dict(T=float("nan")),
            dict(k=torch.tensor([-5, 2 ** 31 - 1, V, V - 1, 1])), dict(p=torch.tensor([-1.0, 0.0, 1e-30, 1.0, INF])),
            dict(q=torch.tensor([-1.0, 1e-30, 1.0, INF, 0.5])), dict(u=0.0),
            dict(u=torch.tensor([-3.0, 0.0, 2.0 ** -24, 1 - 2.0 ** -24, 2.0 ** -60])),
            dict(k=7, u=torch.tensor([1.0, 1.5, INF, -1.0, -INF])))):
        print(f"extreme {kw}", flush=True)
        check(l, seed=50 + i, **kw)
    check(l * 100, seed=60)
    check(normal(3, V, 2.0, 33) * 1e30, seed=61)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("ld", [V, V + 7, V + 1000])
def test_padded_rows(dtype, ld):
    """Rows at any distance and alignment; what lies between them is not read as a logit."""
    t = torch.full((6, ld), 1e4, dtype=dtype)
    t[:, :V] = normal(6, V, 2.0, ld, dtype)
    check(t[:, :V], k=30, p=0.9, seed=3)
    check(t[:, :V], T=1.3, p=0.95, q=0.001, seed=4)


@pytest.mark.parametrize("B,V", [(520, 16385), (700, 17003)])
def test_one_workgroup_per_row(B, V):
    g = torch.Generator().manual_seed(B)
    l = normal(B, V, 2.5, B)
    l[::7, : V // 2] = -INF
    check(l, T=0.3 + torch.rand(B, generator=g), k=torch.randint(0, 200, (B,), generator=g),
          p=0.4 + 0.7 * torch.rand(B, generator=g), q=0.05 * torch.rand(B, generator=g), seed=8)


@pytest.mark.parametrize("value", [-1e4, float(torch.finfo(torch.float32).min), -INF], ids=["1e4", "lowest", "inf"])
def test_flat_rows_under_a_mask(value):
    """Crowded bins where a mask's value is finite: the range of nearly equal logits is narrowed."""
    l = normal(4, V, 0.004, 34)
    l[:, ::3] = value
    check(l, seed=1)
    check(l, p=0.6, seed=2)
    check(l, k=20001, p=0.9, seed=3)
    check(l, q=0.9951, seed=4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_longest_rows(dtype):
    """2^20 tokens, also with all weights equal (their sum is 2^63)."""
    l = normal(3, 1 << 20, 2.0, 35, dtype)
    check(l, T=torch.tensor([0.7, 1.0, 1.5]), k=torch.tensor([0, 50, 100000]), p=torch.tensor([0.9, 1.0, 0.7]),
          seed=5)
    check(l, T=INF, seed=6)
    check(l, T=INF, k=700001, p=0.75, seed=7)


def test_most_rows():
    l = normal(32768, 33, 2.0, 36)
    g = torch.Generator().manual_seed(9)
    check(l, T=0.2 + torch.rand(32768, generator=g), k=torch.randint(0, 40, (32768,), generator=g),
          p=0.3 + 0.8 * torch.rand(32768, generator=g), q=0.05 * torch.rand(32768, generator=g), seed=10)


def test_graphs_of_both_forms_share_a_workspace():
    """The one-launch and the four-launch form captured, replayed in turn over one workspace with new logits."""
    g = torch.Generator().manual_seed(12)
    cases = []
    for B, n in ((5, 9001), (3, V)):
        lg = torch.empty(B, n, device=DEV)
        kw = dict(temperature=torch.full((B,), 0.8, device=DEV), top_p=torch.full((B,), 0.9, device=DEV))
        cases.append((B, n, lg, torch.rand(B, generator=g).to(DEV), torch.empty(B, dtype=torch.int32, device=DEV), kw))
    ws = torch.full((ds4.sample_workspace_bytes(3, V),), 0xA5, dtype=torch.uint8, device=DEV)
    call = lambda c: ds4.sample(c[0], c[1], c[2], c[3], c[4], workspace=ws, **c[5])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in cases:
            c[2].zero_()
            call(c)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(c)
        graphs.append(graph)
    for rep in range(6):
        for c, graph in zip(cases, graphs):
            l = normal(c[0], c[1], 2.0, 70 + rep)
            c[2].copy_(l)
            c[4].fill_(-9)
            ws.fill_(0x5A)
            torch.randn(1000, device=DEV).sum().item()
            graph.replay()
            torch.cuda.synchronize()
            host, u = l.double().numpy(), c[3].cpu()
            T, p = float(torch.tensor(0.8)), float(torch.tensor(0.9))
            for r in range(c[0]):
                assert int(c[4][r]) == reference(host[r], T, 0, p, 0.0, float(u[r]))[0], (rep, r)
