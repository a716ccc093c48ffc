"""ds4moe_linear, ds4moe_grouped_matmul and their gradients refuse bad
arguments on the host, before any launch (no GPU: nothing here reaches one)."""
import ctypes

import pytest

ds4 = pytest.importorskip("bit_routed_moe_amd")

FAKE, MIS, BIG = 0x100000, 0x100004, 1 << 40
c = ctypes.byref


def lin(m, rows=4, x=FAKE, w=FAKE, bias=None, res=None, y=FAKE, z=None, ws=FAKE, n=BIG):
    # an odd pointer stops every otherwise valid call before a launch
    return ds4.lib.ds4moe_linear(m and c(m), rows, x, w, bias, res, y, z, ws, n, None)


def grp(m, rows=4, x=FAKE, x_rows=4, w=FAKE, bias=None, off=FAKE, sp=None, k=1, y=FAKE, z=None, ws=FAKE, n=BIG):
    return ds4.lib.ds4moe_grouped_matmul(c(m), rows, x, x_rows, w, bias, off, sp, k, y, z, ws, n, None)


def bwd(m, rows=4, x=FAKE, w=FAKE, z=FAKE, dy=FAKE, dx=FAKE, dw=FAKE, db=None, ws=FAKE, n=BIG):
    return ds4.lib.ds4moe_linear_backward(c(m), rows, x, w, z, dy, dx, dw, db, ws, n, None)


def gbwd(m, rows=4, x=FAKE, x_rows=4, w=FAKE, z=FAKE, dy=FAKE, off=FAKE, sp=None, k=1, dx=FAKE, dw=FAKE, db=None,
         ws=FAKE, n=BIG):
    return ds4.lib.ds4moe_grouped_matmul_backward(c(m), rows, x, x_rows, w, z, dy, off, sp, k, dx, dw, db, ws, n,
                                                  None)


def test_descriptor():
    mk = ds4.make_matmul
    assert lin(None) == -1
    assert lin(mk(0, 8)) == -2 and lin(mk(8, 0)) == -2
    assert lin(mk((1 << 20) + 8, 8)) == -2 and lin(mk(8, (1 << 20) + 1)) == -2
    assert lin(mk(64, 64), rows=0) == -2 and lin(mk(64, 64), rows=-1) == -2
    assert lin(mk(64, 64), rows=(1 << 24) + 1) == -2
    assert lin(mk(1 << 20, 64), rows=1 << 20) == -2          # more tiles than a launch takes
    assert lin(mk(1 << 20, 1 << 20)) == -2
    assert lin(mk(64, 1 << 20), rows=1 << 16) == -2
    assert grp(mk(64, 1 << 20, groups=1024), rows=4096, x_rows=4096) == -2
    assert grp(mk(64, 1 << 18, groups=1024), rows=4096, x_rows=4096, x=MIS) == -3
    assert lin(mk(64, 64, groups=2)) == -2                   # linear: one group
    assert grp(mk(64, 64, groups=0)) == -2 and grp(mk(64, 64, groups=1025)) == -2
    assert lin(mk(64, 65, act="swiglu")) == -2
    bad = mk(64, 64)
    bad.act = 6
    assert lin(bad) == -1
    bad = mk(64, 64)
    bad.dtype = 2
    assert lin(bad) == -4
    bad.dtype = 7
    assert lin(bad) == -1
    assert lin(mk(64, 64, dtype="f32", grad="bf16")) == -4
    bad = mk(64, 64)
    bad.grad_dtype = 2
    assert lin(bad) == -4


def test_strides():
    mk = ds4.make_matmul
    assert lin(mk(65, 64)) == -2                             # rows of 65 bf16 elements without a stride
    assert lin(mk(64, 65)) == -2
    assert lin(mk(66, 64, dtype="f32")) == -2
    assert lin(mk(64, 64, ldx=56)) == -2 and lin(mk(64, 64, ldx=65)) == -2
    assert lin(mk(64, 64, ldw=68)) == -2 and lin(mk(64, 64, ldy=60)) == -2
    assert lin(mk(64, 64, ldx=-64)) == -2
    assert lin(mk(64, 64, ldz=68), z=FAKE) == -2             # z's stride matters only with z
    assert lin(mk(64, 64, ldz=68), z=None, x=MIS) == -3


def test_pointers():
    m = ds4.make_matmul(64, 64)
    assert lin(m, x=None) == -1 and lin(m, w=None) == -1 and lin(m, y=None) == -1
    for name in ("x", "w", "bias", "res", "y", "z"):
        assert lin(m, **{name: MIS}) == -3, name
    g = ds4.make_matmul(64, 64, groups=3)
    assert grp(g, off=None) == -1 and grp(g, off=MIS) == -3 and grp(g, sp=MIS) == -3
    assert grp(g, x_rows=5) == -2                            # without sorted_pair x has `rows` rows
    assert grp(g, sp=FAKE, k=0) == -2 and grp(g, sp=FAKE, x_rows=0) == -2
    assert bwd(m, dy=None) == -1 and bwd(m, x=None) == -1 and bwd(m, w=None) == -1
    assert bwd(m, dx=None, dw=None) == -1
    assert bwd(ds4.make_matmul(64, 64, act="silu"), z=None) == -1
    for name in ("x", "w", "dy", "dx", "dw", "db"):
        assert bwd(m, **{name: MIS}) == -3, name
    assert gbwd(g, off=None) == -1 and gbwd(g, sp=MIS) == -3


def test_workspace():
    m = ds4.make_matmul(64, 64, groups=3, act="silu")
    for fn, back in ((grp, False), (gbwd, True)):
        need = ds4.matmul_workspace_bytes(m, 4, back)
        assert need > 0
        assert fn(m, ws=None) == -5 and fn(m, n=need - 1) == -5 and fn(m, ws=MIS) == -3
    assert ds4.matmul_workspace_bytes(ds4.make_matmul(0, 64), 4) == 0
    assert ds4.matmul_workspace_bytes(ds4.make_matmul(64, 64), 4) == 0     # dense forward: none
    for act in ("none", "swiglu"):
        for E in (1, 3, 64):
            m = ds4.make_matmul(64, 64, groups=E, act=act)
            for back in (False, True):
                sizes = [ds4.matmul_workspace_bytes(m, r, back) for r in (1, 2, 5, 17, 100, 1000, 5000)]
                assert sizes == sorted(sizes)
