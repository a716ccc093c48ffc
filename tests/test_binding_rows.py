"""Tensors whose memory is not what their shape says: the bindings of the rows'
quantization and of the rules on logits refuse them (no GPU: nothing here
reaches one)."""
import pytest
import torch

ds4 = pytest.importorskip("bit_routed_moe_amd")

I8 = torch.int8


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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_refuses_rows_closer_than_their_columns(lib, dtype):
    """A stride of 0 (one row, broadcast) is no "without gaps", and rows may not overlap."""
    rows, cols = 5, 64
    good = dict(x=torch.zeros(rows, cols, dtype=dtype), codes=torch.zeros(rows, cols, dtype=I8), scale=torch.zeros(rows))
    ds4.quantize_rows_int8(rows, cols, **good)
    assert lib.called.pop()[0] == "ds4moe_quantize_rows_int8"
    for name in ("x", "codes"):
        t = good[name]
        for bad in (t[:1].expand(rows, cols), t[:1, None].expand(rows, 1, cols), t[None, :1].expand(1, rows, cols),
                    t.as_strided((rows, cols), (16, 1)), t[0].expand(2, 3, cols)):
            with pytest.raises(ds4.Ds4MoeError, match=name) as e:
                ds4.quantize_rows_int8(rows, cols, **dict(good, **{name: bad}))
            assert e.value.status == -2 and not lib.called, (name, bad.shape, bad.stride())
    # one row has no stride: any is taken
    ds4.quantize_rows_int8(1, cols, good["x"][:1].expand(rows, cols), good["codes"][:1].expand(rows, cols), good["scale"])
    a = lib.called.pop()[1]
    assert a[4] >= cols and a[6] >= cols


def test_mask_without_rows_is_no_mask_left_out(lib):
    """An empty tensor has no memory; without mask_row its rows are too few, which is not the rule switched off."""
    B, V = 3, 100
    call = lambda **kw: ds4.adjust_logits(B, V, torch.zeros(B, V), torch.zeros(B, V), **kw)
    for words in (4, 9):
        empty = torch.zeros(0, words, dtype=torch.int32)
        with pytest.raises(ds4.Ds4MoeError, match="mask") as e:
            call(mask=empty)
        assert e.value.status == -2 and not lib.called
        call(mask=empty, mask_row=torch.zeros(B, dtype=torch.int32))     # (every row's mask_row is then outside: no mask)
        assert lib.called.pop()[0] == "ds4moe_adjust_logits"
    call(mask=torch.zeros(B, 4, dtype=torch.int32))
    r = lib.called.pop()[1][5]._obj
    assert r.mask and r.mask_rows == B


def test_lists_beyond_their_offsets_reach_are_refused(lib):
    """Offsets are int32: a longer list's length would be passed modulo 2^32, and its rules be left out.  (Tensors
    without memory stand for the 16 GB.)"""
    B, V = 3, 100
    i = lambda *s, **kw: torch.zeros(*s, dtype=torch.int32, **kw)
    good = dict(history=i(9), history_offsets=i(B + 1), bias_token=i(4), bias_value=torch.zeros(4), bias_offsets=i(B + 1))
    call = lambda **kw: ds4.adjust_logits(B, V, torch.zeros(B, V), torch.zeros(B, V), **dict(good, **kw))
    call()
    lib.called.pop()
    for n in (1 << 31, (1 << 32) + 5):
        for kw in (dict(history=i(n, device="meta")),
                   dict(bias_token=i(n, device="meta"), bias_value=torch.zeros(n, device="meta"))):
            with pytest.raises(ds4.Ds4MoeError, match="history|bias_token") as e:
                call(**kw)
            assert e.value.status == -2 and not lib.called
