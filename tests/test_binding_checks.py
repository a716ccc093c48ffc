"""The Python binding refuses tensors that its descriptor or its arguments do
not describe, before the library is called.  No GPU: the library is replaced by
a recorder, and tensors on the host stand for those on the current device."""
import pytest
import torch

ds4 = pytest.importorskip("bit_routed_moe_amd")

ARG, SHAPE = -1, -2


class Recorder:
    """In place of the library: every entry point notes its name and succeeds."""

    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        return lambda *args: self.called.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(ds4, "lib", r)
    monkeypatch.setattr(ds4, "_here", lambda: -1, raising=False)   # (a host tensor's device index)
    monkeypatch.setattr(ds4, "_s", lambda *args: None)
    return r


def refused(lib, status, match, fn, *args, **kw):
    with pytest.raises(ds4.Ds4MoeError, match=match) as e:
        fn(*args, **kw)
    assert e.value.status == status and not lib.called


def accepted(lib, fn, *args, **kw):
    fn(*args, **kw)
    assert len(lib.called) == 1
    lib.called.clear()


# ---- sample ----------------------------------------------------------------------

def sample_args(B=3, V=50):
    a = dict(logits=torch.zeros(B, V), u=torch.zeros(B), token=torch.zeros(B, dtype=torch.int32),
             temperature=torch.ones(B), top_k=torch.ones(B, dtype=torch.int32), top_p=torch.ones(B),
             min_p=torch.zeros(B), prob=torch.zeros(B))
    return B, V, a


def test_sample_types(lib):
    B, V, a = sample_args()
    accepted(lib, ds4.sample, B, V, **a)
    accepted(lib, ds4.sample, B, V, **dict(a, logits=a["logits"].bfloat16()))
    for n in ("temperature", "top_k", "top_p", "min_p", "prob"):
        accepted(lib, ds4.sample, B, V, **dict(a, **{n: None}))
    for n, t in a.items():
        for dt in (torch.int64, torch.float64, torch.float16, torch.int32, torch.float32):
            if dt != t.dtype and not (n == "logits" and dt == torch.float32):
                refused(lib, ARG, f"{n} (is )?{dt}", ds4.sample, B, V, **dict(a, **{n: t.to(dt)}))


def test_sample_sizes(lib):
    B, V, a = sample_args()
    for n, t in a.items():
        if n != "logits":
            refused(lib, SHAPE, n, ds4.sample, B, V, **dict(a, **{n: t[:-1]}))
            refused(lib, SHAPE, n, ds4.sample, B, V, **dict(a, **{n: t[:1].expand(B)}))         # one value in memory
            refused(lib, SHAPE, n, ds4.sample, B, V, **dict(a, **{n: torch.stack([t, t], 1)[:, 0]}))
            accepted(lib, ds4.sample, B, V, **dict(a, **{n: torch.cat([t, t])}))                # room for more rows
            accepted(lib, ds4.sample, B, V, **dict(a, **{n: t[:, None]}))
    for bad in (torch.zeros(B, V - 1), torch.zeros(B - 1, V), torch.zeros(2, 3, V)[:, 0], torch.zeros(1, B, V)):
        refused(lib, SHAPE, "logits", ds4.sample, B, V, **dict(a, logits=bad))
    for good in (torch.zeros(B + 1, V), torch.zeros(B, V + 6)[:, :V], torch.zeros(B, V + 6), torch.zeros(B, 1, V)):
        accepted(lib, ds4.sample, B, V, **dict(a, logits=good))


def test_sample_one_row(lib):
    _, V, a = sample_args(1)
    accepted(lib, ds4.sample, 1, V, **dict(a, logits=torch.zeros(V)))
    accepted(lib, ds4.sample, 1, V, **dict(a, temperature=torch.tensor(0.7)))       # no dimension: one value
    refused(lib, SHAPE, "logits", ds4.sample, 1, V, **dict(a, logits=torch.zeros(V - 1)))
    refused(lib, SHAPE, "logits", ds4.sample, 1, V, **dict(a, logits=torch.zeros(0, V)))
    refused(lib, SHAPE, "logits", ds4.sample, 3, 1, torch.zeros(1), torch.zeros(3), torch.zeros(3, dtype=torch.int32))


# ---- products --------------------------------------------------------------------

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def product(dtype="bf16", grad=None, act="none", groups=None, rows=6, K=24, N=16, pad=0):
    """Descriptor and tensors of a product (rows at `pad` elements behind one another's ends)."""
    t, g = (BF if dtype == "bf16" else F32), (F32 if (grad or dtype) == "f32" else BF)
    E, oc = groups or 1, N // 2 if act == "swiglu" else N
    m = ds4.make_matmul(K, N, groups=E, dtype=dtype, grad=grad, act=act, ldx=K + pad, ldw=K + pad, ldy=oc + pad,
                        ldz=N + pad)
    mk = lambda r, c, dt: torch.zeros(*r, c + pad, dtype=dt)[..., :c]
    a = dict(x=mk((rows,), K, t), w=mk((E, N), K, t), bias=torch.zeros(E, N, dtype=t), y=mk((rows,), oc, t),
             z=mk((rows,), N, t), residual=mk((rows,), oc, t), dy=mk((rows,), oc, t), dx=mk((rows,), K, t),
             dw=mk((E, N), K, g), dbias=torch.zeros(E, N, dtype=g),
             expert_offsets=torch.zeros(E + 1, dtype=I32), sorted_pair=torch.zeros(rows, dtype=I32))
    return m, rows, a


FORWARD = ("x", "w", "y", "bias", "residual", "z")
BACKWARD = ("x", "w", "dy", "z", "dx", "dw", "dbias")
GROUPED = ("x", "w", "expert_offsets", "y", "bias", "z", "sorted_pair")
GROUPED_BACKWARD = ("x", "w", "expert_offsets", "dy", "z", "dx", "dw", "dbias", "sorted_pair")
CALLS = [("linear", FORWARD, None), ("linear_backward", BACKWARD, None), ("grouped_matmul", GROUPED, 3),
         ("grouped_matmul_backward", GROUPED_BACKWARD, 3)]


def pick(a, names):
    return {n: a[n] for n in names}


@pytest.mark.parametrize("fn,names,groups", CALLS, ids=[c[0] for c in CALLS])
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_product_types(lib, fn, names, groups, dtype, grad):
    m, rows, a = product(dtype, grad, "silu", groups)
    call, a = getattr(ds4, fn), pick(a, names)
    accepted(lib, call, m, rows, **a)
    for n, t in a.items():
        for dt in (torch.int64, torch.float64, torch.float16, torch.int32, torch.float32, torch.bfloat16):
            if dt != t.dtype:
                refused(lib, ARG, f"{n} is {dt}", call, m, rows, **dict(a, **{n: t.to(dt)}))
