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


@pytest.mark.parametrize("fn,names,groups", CALLS, ids=[c[0] for c in CALLS])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_product_sizes_and_strides(lib, fn, names, groups, act):
    vectors = ("bias", "dbias", "expert_offsets", "sorted_pair")
    for pad in (0, 8):
        m, rows, a = product("bf16", "f32", act, groups, pad=pad)
        call, a = getattr(ds4, fn), pick(a, names)
        accepted(lib, call, m, rows, **a)
        for n, t in a.items():
            cols, last = t.shape[-1], t.dim() - 1
            if n in vectors:
                flat = t.flatten()
                bad = [flat[:-1], flat[:1].expand(flat.numel()), torch.stack([flat, flat], 1)[:, 0]]
                good = [flat, torch.cat([flat, flat])]
            else:
                r = t.numel() // cols
                # a row or a column too few; a row stride that is not the descriptor's; columns apart
                bad = [t.narrow(t.dim() - 2, 0, t.shape[-2] - 1), t.narrow(last, 0, cols - 1),
                       torch.zeros(*t.shape[:-1], cols + 16, dtype=t.dtype)[..., :cols],
                       torch.zeros(*t.shape, 2, dtype=t.dtype)[..., 0],
                       torch.zeros((r - 1) * (cols + pad) + cols - 1, dtype=t.dtype)]
                if t.dim() == 3 and groups:     # experts that do not follow one another at out_dim rows
                    bad.append(torch.zeros(t.shape[0], t.shape[1] + 1, cols + pad, dtype=t.dtype)[:, :-1, :cols])
                whole = torch.zeros(r, cols + pad, dtype=t.dtype)
                good = [whole, whole[:, :cols], whole.flatten(), torch.zeros(r // 2, 2, cols + pad, dtype=t.dtype)]
                if n != "x" or fn.startswith("linear"):     # (x's rows are part of the grouped calls)
                    good.append(torch.zeros(r + 3, cols + pad, dtype=t.dtype))
            kw = {"x_rows": rows} if groups else {}
            for b in bad:
                refused(lib, SHAPE, f"{n} of shape", call, m, rows, **dict(a, **{n: b}), **kw)
            for b in good:
                accepted(lib, call, m, rows, **dict(a, **{n: b}), **kw)


def test_product_unread_operands(lib):
    """x is read for dw only, w for dx only, z for an activation only: otherwise they may be anything."""
    m, rows, a = product(act="none")
    accepted(lib, ds4.linear_backward, m, rows, None, a["w"], a["dy"], z=torch.zeros(1), dx=a["dx"])
    accepted(lib, ds4.linear_backward, m, rows, a["x"], None, a["dy"], dw=a["dw"])
    accepted(lib, ds4.linear_backward, m, rows, torch.zeros(1), torch.zeros(1), a["dy"], dbias=a["dbias"])


def test_product_row_counts(lib):
    """x's rows: as many as x_rows says (default: all of its leading dimensions); one row has no stride."""
    m, rows, a = product(groups=3)
    call = lambda **kw: ds4.grouped_matmul(m, rows, **dict(pick(a, GROUPED), **kw))
    refused(lib, SHAPE, "x of shape", call, x_rows=rows + 1)
    seen = []
    lib.__class__ = type("R", (Recorder,), {"__getattr__": lambda self, n: lambda *args: seen.append(args[3]) or 0})
    call(x=torch.zeros(2, 5, 24, dtype=BF))
    call(x=torch.zeros(4, 24, dtype=BF))
    call(x=torch.zeros(24 * 7, dtype=BF), x_rows=7)
    assert seen == [10, 4, 7]
    lib.__class__ = Recorder
    m, rows, a = product(rows=1)
    accepted(lib, ds4.linear, m, 1, torch.zeros(3, 40, dtype=BF)[:1, :24], a["w"], a["y"])
    accepted(lib, ds4.linear, m, 1, torch.zeros(24, dtype=BF), a["w"], torch.zeros(16, dtype=BF))


def test_workspace_with_gaps(lib):
    """Bytes between a workspace's elements (or the same ones counted again) are not scratch."""
    m, rows, a = product()
    for ws in (torch.zeros(64, 2, dtype=torch.uint8)[:, 0], torch.zeros(1, dtype=torch.uint8).expand(4096)):
        refused(lib, SHAPE, "workspace", ds4.linear, m, rows, **pick(a, FORWARD), workspace=ws)
        B, V, b = sample_args()
        refused(lib, SHAPE, "workspace", ds4.sample, B, V, **b, workspace=ws)
    accepted(lib, ds4.linear, m, rows, **pick(a, FORWARD), workspace=torch.zeros(8, 8))


def test_product_empty_and_strided_memory(lib):
    """A tensor without elements has no row, and memory without rows has no gaps."""
    m, _, a = product(rows=1)
    w, y = a["w"], a["y"]
    for bad in (torch.zeros(0, 24, dtype=BF), torch.zeros(0, 1, 24, dtype=BF), torch.zeros(1, 0, 24, dtype=BF)):
        refused(lib, SHAPE, "x of shape", ds4.linear, m, 1, bad, w, y)
    m = ds4.make_matmul(1, 16, ldx=8, ldw=8)
    w = torch.zeros(16, 8, dtype=BF)[:, :1]
    accepted(lib, ds4.linear, m, 2, torch.zeros(9, dtype=BF), w, torch.zeros(2, 16, dtype=BF))
    accepted(lib, ds4.linear, m, 2, torch.zeros(2, 8, dtype=BF)[:, :1], w, torch.zeros(2, 16, dtype=BF))
    x = torch.zeros(18, dtype=BF)[::2]
    refused(lib, SHAPE, "x of shape", ds4.linear, m, 2, x, w, torch.zeros(2, 16, dtype=BF))
