"""ds4moe_dispatch, ds4moe_collect, their gradients and ds4moe_route_backward
refuse bad arguments on the host before any launch, and the binding refuses
tensors that its descriptor does not describe (no GPU: nothing here reaches
one)."""
import ctypes

import pytest
import torch

ds4 = pytest.importorskip("bit_routed_moe_amd")

FAKE, MIS = 0x100000, 0x100004
c = ctypes.byref
L = ds4.lib


def dispatch(d, T=4, rows=8, x=FAKE, pos=FAKE, w=None, sp=None, out=FAKE):
    return L.ds4moe_dispatch(d and c(d), T, rows, x, pos, w, sp, out, None)


def collect(d, T=4, rows=8, x=FAKE, pos=FAKE, w=None, base=None, out=FAKE):
    return L.ds4moe_collect(d and c(d), T, rows, x, pos, w, base, out, None)


def dispatch_bwd(d, T=4, rows=8, x=FAKE, dout=FAKE, pos=FAKE, w=None, out=FAKE, dw=FAKE):
    return L.ds4moe_dispatch_backward(d and c(d), T, rows, x, dout, pos, w, out, dw, None)


def collect_bwd(d, T=4, rows=8, x=FAKE, dy=FAKE, pos=FAKE, w=None, sp=None, out=FAKE, dw=FAKE):
    return L.ds4moe_collect_backward(d and c(d), T, rows, x, dy, pos, w, sp, out, dw, None)


ALL = [dispatch, collect, dispatch_bwd, collect_bwd]


@pytest.mark.parametrize("f", ALL)
def test_descriptor(f):
    mk = ds4.make_rows
    assert f(None) == -1
    assert f(mk(0, 2)) == -2 and f(mk((1 << 20) + 8, 2)) == -2
    assert f(mk(64, 0)) == -2 and f(mk(64, 65)) == -2
    assert f(mk(64, 2), T=0) == -2 and f(mk(64, 2), T=(1 << 20) + 1) == -2
    assert f(mk(64, 2), rows=0) == -2 and f(mk(64, 2), rows=-1) == -2
    bad = mk(64, 2)
    bad.dtype = 2
    assert f(bad) == -4
    bad.dtype = 9
    assert f(bad) == -1
    assert f(mk(65, 2)) == -2 and f(mk(66, 2, "f32")) == -2          # rows off 16-byte boundaries
    assert f(mk(64, 2, ldx=56)) == -2 and f(mk(64, 2, ldr=68)) == -2 and f(mk(64, 2, ldr=-64)) == -2
    assert f(mk(64, 2, ldx=(1 << 31) + 8)) == -2
    for name in ("x", "pos", "w", "out"):
        assert f(mk(64, 2), **{name: MIS}) == -3, name
    assert f(mk(64, 2), x=None) == -1 and f(mk(64, 2), pos=None) == -1


def test_pointers():
    d = ds4.make_rows(64, 2)
    assert dispatch(d, out=None) == -1 and collect(d, out=None) == -1
    assert dispatch(d, sp=MIS) == -3 and collect_bwd(d, sp=MIS) == -3 and collect(d, base=MIS) == -3
    assert dispatch_bwd(d, dout=None) == -1 and collect_bwd(d, dy=None) == -1
    assert dispatch_bwd(d, dout=MIS) == -3 and collect_bwd(d, dy=MIS) == -3
    for f in (dispatch_bwd, collect_bwd):
        assert f(d, out=None, dw=None) == -1 and f(d, dw=MIS) == -3
        assert f(d, x=None, dw=None, pos=None) == -1                 # x is read for dtopk_w only


def test_route_backward_arguments():
    f = L.ds4moe_route_backward
    cfg = ds4.make_config(256, 128, 8, 2)
    assert f(None, 4, FAKE, FAKE, FAKE, FAKE, None) == -1
    assert f(c(ds4.make_config(256, 128, 8, 9)), 4, FAKE, FAKE, FAKE, FAKE, None) == -2
    assert f(c(cfg), 0, FAKE, FAKE, FAKE, FAKE, None) == -2
    for i in range(4):
        p = [FAKE] * 4
        p[i] = None
        assert f(c(cfg), 4, *p, None) == -1
        p[i] = MIS
        assert f(c(cfg), 4, *p, None) == -3


class Recorder:
    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        return lambda *args: self.called.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(ds4, "lib", r)
    monkeypatch.setattr(ds4, "_here", lambda: -1)
    monkeypatch.setattr(ds4, "_s", lambda *args: None)
    return r


T, K, H, R = 5, 3, 24, 11
I32, F32, BF = torch.int32, torch.float32, torch.bfloat16
TENSORS = dict(x=(T, H), y=(T, H), dx=(T, H), dy=(T, H), base=(T, H), out=(R, H), dout=(R, H), expert_rows=(R, H),
               drows=(R, H), topk_w=(T, K), dtopk_w=(T, K), pair_pos=(T * K,), sorted_pair=(R,))
CALLS = {"dispatch": ("x", "pair_pos", "out", "topk_w", "sorted_pair"),
         "collect": ("expert_rows", "pair_pos", "y", "topk_w", "base"),
         "dispatch_backward": ("dout", "pair_pos", "topk_w", "x", "dx", "dtopk_w"),
         "collect_backward": ("dy", "pair_pos", "expert_rows", "topk_w", "sorted_pair", "drows", "dtopk_w")}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fn", CALLS)
def test_binding_refuses(lib, fn, dtype):
    row_type = BF if dtype == "bf16" else F32

    def made(n):
        t = I32 if n in ("pair_pos", "sorted_pair") else F32 if n.endswith("topk_w") else row_type
        return torch.zeros(TENSORS[n], dtype=t)

    d = ds4.make_rows(H, K, dtype)
    good = {n: made(n) for n in CALLS[fn]}

    def refused(status, match, **change):
        with pytest.raises(ds4.Ds4MoeError, match=match) as e:
            getattr(ds4, fn)(d, T, R, **dict(good, **change))
        assert e.value.status == status and not lib.called

    def accepted(**change):
        getattr(ds4, fn)(d, T, R, **dict(good, **change))
        assert lib.called == ["ds4moe_" + fn]
        lib.called.clear()

    accepted()
    for n, t in good.items():
        for other in (torch.int64, torch.float64, torch.float16, I32, F32, BF):
            if other != t.dtype:
                refused(-1, n, **{n: t.to(other)})
        refused(-2, n, **{n: t.reshape(-1)[:-1]} if t.dim() == 1 or n.endswith("topk_w") else {n: t[:-1]})
        if t.dim() == 2 and not n.endswith("topk_w"):
            refused(-2, n, **{n: t[:, :-1]})
            refused(-2, n, **{n: torch.zeros(t.shape[0], H + 8, dtype=t.dtype)[:, :H]})
            accepted(**{n: torch.zeros(t.shape[0] + 2, H, dtype=t.dtype)})
        refused(-2, n, **{n: torch.stack([t, t], -1)[..., 0]})
    for n in ("topk_w", "sorted_pair", "base"):
        if n in good:
            accepted(**{n: None})


def test_binding_route_backward(lib):
    cfg = ds4.make_config(256, 128, 8, K)
    good = dict(topk_idx=torch.zeros(T, K, dtype=I32), topk_w=torch.zeros(T, K), dtopk_w=torch.zeros(T, K),
                dlogits=torch.zeros(T, 8))
    ds4.route_backward(cfg, T, **good)
    assert lib.called == ["ds4moe_route_backward"]
    lib.called.clear()
    for n, t in good.items():
        for bad, st in ((t.double(), -1), (t[:-1], -2), (t.t().contiguous().t(), -2)):
            with pytest.raises(ds4.Ds4MoeError, match=n) as e:
                ds4.route_backward(cfg, T, **dict(good, **{n: bad}))
            assert e.value.status == st and not lib.called


def test_other_devices_are_refused(monkeypatch):
    """Tensors on the host (or another device) while device 0 is current."""
    monkeypatch.setattr(ds4, "lib", Recorder())
    monkeypatch.setattr(ds4, "_here", lambda: 0)
    monkeypatch.setattr(ds4, "_s", lambda *args: None)
    d, cfg = ds4.make_rows(H, K), ds4.make_config(256, 128, 8, K)
    m = ds4.make_matmul_int8(32, 16, groups=1)
    row = lambda n, w=H, t=BF: torch.zeros(n, w, dtype=t)
    i32 = lambda n: torch.zeros(n, dtype=I32)
    i8 = lambda n: torch.zeros(n, 32, dtype=torch.int8)
    f = torch.zeros
    for call in (lambda: ds4.dispatch(d, T, R, row(T), i32(T * K), row(R)),
                 lambda: ds4.collect(d, T, R, row(R), i32(T * K), row(T)),
                 lambda: ds4.dispatch_backward(d, T, R, row(R), i32(T * K), dx=row(T)),
                 lambda: ds4.collect_backward(d, T, R, row(T), i32(T * K), drows=row(R)),
                 lambda: ds4.route_backward(cfg, T, i32(T * K), f(T * K), f(T * K), f(T * 8)),
                 lambda: ds4.quantize_rows_int8(4, 32, row(4, 32), i8(4), f(4)),
                 lambda: ds4.linear_int8(m, 4, i8(4), f(4), i8(16), f(16), row(4, 16)),
                 lambda: ds4.grouped_matmul_int8(m, 4, i8(4), f(4), i8(16), f(16), i32(2), row(4, 16)),
                 lambda: ds4.adjust_logits(2, 50, f(2, 50), f(2, 50), bias_token=i32(1), bias_value=f(1), bias_offsets=i32(3))):
        with pytest.raises(ds4.Ds4MoeError, match="not on the current HIP device") as e:
            call()
        assert e.value.status == -1 and not ds4.lib.called
