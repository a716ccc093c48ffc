"""Gradients of the router's weights, logits and the experts' rows against
central differences of the calls themselves, at logits so far apart that the
choice of experts and its order cannot change on the way."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ds4 = pytest.importorskip("bit_routed_moe_amd")
from helpers import DEV  # noqa: E402

H_STEP = 2.0 ** -6


@pytest.mark.parametrize("T,E,k,H", [(6, 12, 4, 40), (3, 9, 8, 129), (17, 40, 2, 7)])
def test_gradients_against_differences(T, E, k, H):
    """L(s) = sum dy * collect(rows + s r, softmax of the chosen logits + s v), |v| <= 1.  With a_j = <rows_j, dy> and
    b_j = <r_j, dy> at token t, L = sum_t sum_j w_j (a_j + s b_j).  Derivatives of w_j by s: its own times v_j - mean(v)
    and so on, |w''| <= 5 w and |w'''| <= 22 w for |v| <= 1 (mean, variance and third moment of v under w are at most 1,
    1 and 8), so the difference is off by h^2 / 6 of max_j 22 |a| + 15 |b| summed over the tokens (a quarter more where
    rows move).  One evaluation in fp32 is off by at most (k + 8) 2^-23 of sum w |rows| |dy|, divided by h; the
    gradients themselves by less."""
    g = torch.Generator().manual_seed(T + E)
    cfg = ds4.make_config(256, 128, E, k)
    d = ds4.make_rows(H, k, "f32", ldr=(H + 3) // 4 * 4, ldx=(H + 3) // 4 * 4)
    ld = (H + 3) // 4 * 4
    # logits a quarter apart, in another order for each token; steps move them by 2^-6 at most
    order = torch.stack([torch.randperm(E, generator=g) for _ in range(T)])
    logits = (order.float() * 0.25).to(DEV)

    def mat(n):
        t = torch.full((n, ld), float("nan"), device=DEV)
        t[:, :H] = torch.empty(n, H).normal_(generator=g).to(DEV)
        return t[:, :H]

    def free(n):
        return torch.empty(n, ld, device=DEV)[:, :H]

    rows, dy = mat(T * k), mat(T)
    pos = torch.randperm(T * k, generator=g).to(torch.int32).to(DEV)
    idx, w, y = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV), free(T)

    def loss(lg, r):
        ds4.route(cfg, T, lg, idx, w)
        ds4.collect(d, T, T * k, r, pos, y, topk_w=w)
        return float((y.double() * dy.double()).sum()), idx.clone()

    _, chosen = loss(logits, rows)
    w0 = w.clone().double()
    drows, dw, dl = free(T * k), torch.empty(T, k, device=DEV), torch.empty(T, E, device=DEV)
    ds4.collect_backward(d, T, T * k, dy, pos, expert_rows=rows, topk_w=w, drows=drows, dtopk_w=dw)
    ds4.route_backward(cfg, T, idx, w, dw, dl)
    at = pos.long().view(T, k)
    dots = lambda m: (m.double()[at] * dy.double()[:, None]).sum(2)
    weight = lambda m: float((w0[:, :, None] * m.double()[at].abs() * dy.double()[:, None].abs()).sum())
    h = H_STEP
    for _ in range(4):
        v = (torch.rand(T, E, generator=g) * 2 - 1).to(DEV)
        v = torch.zeros_like(v).scatter_(1, chosen.long(), v.gather(1, chosen.long()))
        r = mat(T * k)
        there, back = rows.clone(), rows.clone()
        there += h * r
        back -= h * r
        (a, ca), (b, cb) = loss(logits + h * v, padded(there, ld)), loss(logits - h * v, padded(back, ld))
        assert torch.equal(ca, chosen) and torch.equal(cb, chosen)
        want = float((dl.double() * v.double()).sum() + (drows.double() * r.double()).sum())
        third = float((22 * dots(rows).abs() + 15 * dots(r).abs()).amax(1).sum()) * 1.25
        tol = h * h / 6 * third + (k + 8) * 2.0 ** -23 * 2 * (weight(rows) + weight(r)) / h
        size = float((dl.double() * v.double()).norm() + (drows.double() * r.double()).norm())
        assert tol <= 0.05 * size                # (a bound that would catch a wrong term)
        assert abs((a - b) / (2 * h) - want) <= tol, ((a - b) / (2 * h), want, tol)


def padded(t, ld):
    out = torch.full((t.shape[0], ld), float("nan"), device=t.device)
    out[:, :t.shape[1]] = t
    return out[:, :t.shape[1]]
