"""ds4moe_adjust_logits refuses bad arguments on the host before any launch,
and its binding tensors that the call would misread (no GPU: nothing here
reaches one)."""
import ctypes

import pytest
import torch

ds4 = pytest.importorskip("bit_routed_moe_amd")

FAKE, MIS = 0x100000, 0x100004
POINTERS = ("history", "history_offsets", "prompt_len", "repetition", "presence", "frequency", "bias_token",
            "bias_value", "bias_offsets", "mask", "mask_row")


def rules(**kw):
    r = ds4.LogitRules(**{n: FAKE for n in POINTERS}, mask_ld=0, n_history=10, n_bias=3, mask_rows=4)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def call(r, B=2, V=100, logits=FAKE, ld=100, dt=0, out=FAKE + 4096, ldo=100, odt=0):
    return ds4.lib.ds4moe_adjust_logits(B, V, logits, ld, dt, r if r is None else ctypes.byref(r), out, ldo, odt, None)


def test_sizes_and_types():
    r = rules()
    assert call(None) == -1
    assert call(r, B=0) == -2 and call(r, B=32769) == -2
    assert call(r, V=0) == -2 and call(r, V=(1 << 20) + 1, ld=1 << 21, ldo=1 << 21) == -2
    assert call(r, ld=99) == -2 and call(r, ldo=99) == -2 and call(r, ldo=(1 << 31) + 1) == -2
    assert call(r, dt=2) == -4 and call(r, odt=2) == -4 and call(r, dt=3) == -1 and call(r, odt=-1) == -1
    assert call(r, logits=None) == -1 and call(r, out=None) == -1
    assert call(r, logits=MIS) == -3 and call(r, out=MIS) == -3
    assert call(r, out=FAKE, odt=1) == -1                    # in place with another type or stride
    assert call(r, out=FAKE, ldo=104) == -1


def test_rules():
    for n in POINTERS:
        assert call(rules(**{n: MIS})) == -3, n
    for n in ("history_offsets", "bias_value", "bias_offsets"):
        assert call(rules(**{n: None})) == -1, n
    assert call(rules(n_history=-1)) == -2 and call(rules(n_bias=-1)) == -2 and call(rules(mask_rows=-1)) == -2
    assert call(rules(mask_ld=3)) == -2 and call(rules(mask_ld=-4)) == -2
    assert call(rules(mask_row=None, mask_rows=1)) == -2     # without mask_row every row has its own


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


B, V = 3, 100


def tensors():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    return dict(logits=torch.zeros(B, V), out=torch.zeros(B, V), history=i(9), history_offsets=i(B + 1), prompt_len=i(B),
                repetition=torch.ones(B), presence=torch.ones(B), frequency=torch.ones(B), bias_token=i(4),
                bias_value=torch.zeros(4), bias_offsets=i(B + 1), mask=i(2, 4), mask_row=i(B))


def test_binding_refuses(lib):
    good = tensors()

    def refused(status, match, **change):
        with pytest.raises(ds4.Ds4MoeError, match=match) as e:
            ds4.adjust_logits(B, V, **dict(good, **change))
        assert e.value.status == status and not lib.called

    def accepted(**change):
        ds4.adjust_logits(B, V, **dict(good, **change))
        name, args = lib.called.pop()
        assert name == "ds4moe_adjust_logits" and not lib.called
        return args

    accepted()
    for n, t in good.items():
        for other in (torch.int64, torch.float64, torch.float16, torch.int32, torch.float32):
            if other != t.dtype and not (n in ("logits", "out") and other == torch.float32):
                refused(-1, n, **{n: t.to(other)})
        if n not in ("logits", "out"):
            accepted(**{n: None}) if n not in ("history", "bias_token", "mask") else None
        if t.dim() == 1 and n not in ("history", "bias_token"):
            refused(-2, n, **{n: t[:-1]})
        refused(-2, n, **{n: torch.stack([t, t], -1)[..., 0]})
    for n in ("logits", "out"):
        refused(-2, n, **{n: good[n][:, :-1]})
        refused(-2, n, **{n: good[n][:-1]})
        accepted(**{n: torch.zeros(B + 1, V + 7)[:, :V]})
        accepted(**{n: torch.zeros(B, V, dtype=torch.bfloat16)})
    refused(-2, "mask", mask=good["mask"][:, :3])
    refused(-2, "mask", mask=good["mask"][0])
    refused(-2, "mask", mask=good["mask"][:1].expand(2, 4))            # one row in memory
    accepted(mask=torch.zeros(2, 9, dtype=torch.int32)[:, 2:6])


def test_binding_passes_sizes(lib):
    good = tensors()
    good["mask"] = torch.zeros(2, 9, dtype=torch.int32)[:, :4]
    good["logits"] = torch.zeros(B, V + 4, dtype=torch.bfloat16)[:, :V]
    ds4.adjust_logits(B, V, **good)
    args = lib.called.pop()[1]
    assert args[0] == B and args[1] == V and args[3] == V + 4 and args[4] == 1 and args[7] == V and args[8] == 0
    r = args[5]._obj
    assert (r.n_history, r.n_bias, r.mask_rows, r.mask_ld) == (9, 4, 2, 9)
