"""The products in 8-bit integers and the rows' quantization refuse bad
arguments on the host before any launch, and their binding tensors that the
descriptor does not describe (no GPU: nothing here reaches one)."""
import ctypes

import pytest
import torch

ds4 = pytest.importorskip("bit_routed_moe_amd")

FAKE, MIS, BIG = 0x100000, 0x100004, 1 << 40
c = ctypes.byref
L = ds4.lib


def lin(m, rows=4, x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, bias=None, res=None, y=FAKE, wk=FAKE, n=BIG):
    return L.ds4moe_linear_int8(m and c(m), rows, x, xs, w, ws, bias, res, y, wk, n, None)


def grp(m, rows=4, x=FAKE, xs=FAKE, x_rows=4, w=FAKE, ws=FAKE, bias=None, off=FAKE, sp=None, k=1, y=FAKE, wk=FAKE,
        n=BIG):
    return L.ds4moe_grouped_matmul_int8(m and c(m), rows, x, xs, x_rows, w, ws, bias, off, sp, k, y, wk, n, None)


def test_descriptor():
    mk = ds4.make_matmul_int8
    assert lin(None) == -1 and grp(None) == -1
    assert lin(mk(0, 8)) == -2 and lin(mk(8, 0)) == -2
    assert lin(mk(131072, 8)) == -2 and lin(mk(131071, 8, ldx=131072, ldw=131072), x=MIS) == -3
    assert lin(mk(64, (1 << 20) + 1)) == -2
    assert lin(mk(64, 64), rows=0) == -2 and lin(mk(64, 64), rows=(1 << 24) + 1) == -2
    assert lin(mk(64, 64, groups=2)) == -2
    assert grp(mk(64, 64, groups=0)) == -2 and grp(mk(64, 64, groups=1025)) == -2
    assert lin(mk(64, 65, act="swiglu")) == -2
    assert lin(mk(64, 1 << 20), rows=1 << 16) == -2          # more tiles than a launch takes
    for field, value, status in (("act", 6, -1), ("act", -1, -1), ("dtype", 2, -4), ("dtype", 5, -1)):
        bad = mk(64, 64)
        setattr(bad, field, value)
        assert lin(bad) == status


def test_strides_and_pointers():
    mk = ds4.make_matmul_int8
    assert lin(mk(72, 64)) == -2                             # rows of 72 bytes without a stride
    assert lin(mk(64, 68)) == -2 and lin(mk(64, 66, dtype="f32")) == -2
    assert lin(mk(64, 64, ldx=48)) == -2 and lin(mk(64, 64, ldx=72)) == -2 and lin(mk(64, 64, ldw=-64)) == -2
    assert lin(mk(64, 64, ldy=60)) == -2
    m, g = mk(64, 64), mk(64, 64, groups=3)
    for name in ("x", "xs", "w", "ws", "y"):
        assert lin(m, **{name: None}) == -1 and lin(m, **{name: MIS}) == -3, name
        assert grp(g, **{name: None}) == -1 and grp(g, **{name: MIS}) == -3, name
    assert lin(m, bias=MIS) == -3 and lin(m, res=MIS) == -3 and grp(g, bias=MIS) == -3
    assert grp(g, off=None) == -1 and grp(g, off=MIS) == -3 and grp(g, sp=MIS) == -3
    assert grp(g, x_rows=5) == -2 and grp(g, sp=FAKE, k=0) == -2 and grp(g, sp=FAKE, x_rows=0) == -2


def test_workspace():
    g = ds4.make_matmul_int8(64, 64, groups=3)
    need = ds4.matmul_int8_workspace_bytes(g, 4)
    assert need > 0
    assert grp(g, wk=None) == -5 and grp(g, n=need - 1) == -5 and grp(g, wk=MIS) == -3
    assert ds4.matmul_int8_workspace_bytes(ds4.make_matmul_int8(0, 64), 4) == 0
    for E in (1, 3, 64):
        for K in (64, 8192):
            m = ds4.make_matmul_int8(K, 512, groups=E)
            sizes = [ds4.matmul_int8_workspace_bytes(m, r) for r in (1, 2, 5, 17, 100, 1000, 5000)]
            assert sizes == sorted(sizes)


def test_quantize_arguments():
    def q(rows=4, cols=64, dt=0, x=FAKE, ldx=0, codes=FAKE, ldq=0, scale=FAKE):
        return L.ds4moe_quantize_rows_int8(rows, cols, dt, x, ldx, codes, ldq, scale, None)
    assert q(rows=0) == -2 and q(rows=(1 << 24) + 1) == -2 and q(cols=0) == -2 and q(cols=(1 << 20) + 16) == -2
    assert q(dt=2) == -4 and q(dt=3) == -1
    assert q(cols=68) == -2 and q(cols=65, ldx=68) == -2     # codes' rows off 16-byte boundaries
    assert q(ldx=66) == -2 and q(ldx=60) == -2 and q(ldq=72) == -2 and q(ldx=-64) == -2 and q(dt=1, ldx=68) == -2
    for n in ("x", "codes", "scale"):
        assert q(**{n: None}) == -1 and q(**{n: MIS}) == -3


class Recorder:
    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        return lambda *args: self.called.append((name, args)) or 0


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(ds4, "lib", r)
    monkeypatch.setattr(ds4, "_here", lambda: -1)
    monkeypatch.setattr(ds4, "_s", lambda *args: None)
    return r


I8, I32, F32, BF = torch.int8, torch.int32, torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("grouped", [False, True])
def test_binding_refuses(lib, grouped, dtype):
    rows, K, N, E = 6, 32, 16, 3 if grouped else 1
    t = BF if dtype == "bf16" else F32
    m = ds4.make_matmul_int8(K, N, groups=E, dtype=dtype)
    good = dict(x=torch.zeros(rows, K, dtype=I8), x_scale=torch.zeros(rows), w=torch.zeros(E, N, K, dtype=I8),
                w_scale=torch.zeros(E, N), y=torch.zeros(rows, N, dtype=t), bias=torch.zeros(E, N, dtype=t))
    if grouped:
        good |= dict(expert_offsets=torch.zeros(E + 1, dtype=I32), sorted_pair=torch.zeros(rows, dtype=I32))
    else:
        good |= dict(residual=torch.zeros(rows, N, dtype=t))
    fn = ds4.grouped_matmul_int8 if grouped else ds4.linear_int8

    def refused(status, match, **change):
        with pytest.raises(ds4.Ds4MoeError, match=match) as e:
            fn(m, rows, **dict(good, **change))
        assert e.value.status == status and not lib.called

    fn(m, rows, **good)
    assert lib.called.pop()[0] == ("ds4moe_grouped_matmul_int8" if grouped else "ds4moe_linear_int8")
    for n, v in good.items():
        for other in (torch.int64, torch.float64, I8, I32, F32, BF):
            if other != v.dtype:
                refused(-1, n, **{n: v.to(other)})
        if not (grouped and n == "x"):       # (x's rows are counted; x_scale then is too long, not x too short)
            refused(-2, n, **{n: v.reshape(-1, v.shape[-1])[:-1] if v.dim() > 1 else v[:-1]})
        refused(-2, n, **{n: torch.stack([v, v], -1)[..., 0]})
    refused(-2, "workspace", workspace=torch.zeros(4, 4)[:, 0])


def test_binding_quantize(lib):
    good = dict(x=torch.zeros(5, 30)[:, :20], codes=torch.zeros(5, 48, dtype=I8)[:, :20], scale=torch.zeros(5))
    ds4.quantize_rows_int8(5, 20, **good)
    name, a = lib.called.pop()
    assert name == "ds4moe_quantize_rows_int8" and a[:3] == (5, 20, 0) and a[4] == 30 and a[6] == 48
    ds4.quantize_rows_int8(5, 20, **dict(good, x=good["x"].bfloat16()))
    assert lib.called.pop()[1][2] == 1
    ds4.quantize_rows_int8(1, 20, torch.zeros(24), torch.zeros(32, dtype=I8), torch.zeros(1))
    a = lib.called.pop()[1]
    assert a[4] % 8 == 0 and a[6] % 16 == 0
    for change, st in ((dict(x=torch.zeros(5, 20, dtype=torch.float64)), -1), (dict(x=torch.zeros(5, 19)), -2),
                       (dict(x=torch.zeros(4, 20)), -2), (dict(codes=torch.zeros(5, 20, dtype=torch.uint8)), -1),
                       (dict(codes=torch.zeros(4, 32, dtype=I8)), -2), (dict(scale=torch.zeros(4)), -2),
                       (dict(scale=torch.zeros(5, dtype=torch.float64)), -1), (dict(x=torch.zeros(20, 5).t()), -2)):
        with pytest.raises(ds4.Ds4MoeError) as e:
            ds4.quantize_rows_int8(5, 20, **dict(good, **change))
        assert e.value.status == st and not lib.called
