"""ds4moe_sample refuses bad arguments on the host, before any launch."""
import pytest

ds4 = pytest.importorskip("bit_routed_moe_amd")

FAKE, MIS, BIG = 0x100000, 0x100004, 1 << 40


def call(B=2, V=100, logits=FAKE, ld=100, dtype=0, t=None, k=None, p=None, q=None, u=FAKE, token=FAKE, prob=None,
         ws=FAKE, n=BIG):
    return ds4.lib.ds4moe_sample(B, V, logits, ld, dtype, t, k, p, q, u, token, prob, ws, n, None)


def test_refusals():
    assert call(B=0) == -2 and call(B=32769) == -2 and call(B=-1) == -2
    assert call(V=0) == -2 and call(V=(1 << 20) + 1, ld=1 << 21) == -2
    assert call(ld=99) == -2 and call(ld=-100) == -2 and call(ld=(1 << 31) + 1) == -2
    assert call(dtype=2) == -4 and call(dtype=3) == -1 and call(dtype=-1) == -1
    assert call(logits=None) == -1 and call(u=None) == -1 and call(token=None) == -1
    for name in ("logits", "t", "k", "p", "q", "u", "token", "prob"):
        assert call(**{name: MIS}) == -3, name


def test_workspace_sizes():
    assert ds4.sample_workspace_bytes(0, 100) == 0 and ds4.sample_workspace_bytes(1, 0) == 0
    for B, V in ((1, 1000), (1, 131072), (64, 131072)):
        need = ds4.sample_workspace_bytes(B, V)
        if need:
            assert call(B=B, V=V, ld=V, ws=None) == -5 and call(B=B, V=V, ld=V, n=need - 1) == -5
