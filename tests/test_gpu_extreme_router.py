"""Values of the router's gradient at extreme logits: rows whose largest logit
lies on either side of where the sigmoids are taken relative to it, masks of the
lowest value and -inf, wide rows; the balance and the routed part, and the bias."""
import pytest
import torch

import expert_reference as ref
from combine_moe_dispatch_amd import api

pytestmark = pytest.mark.gpu

COEF, UP = 0.5, 0.75
LOWEST = torch.finfo(torch.float32).min
TOPS = [-63.5, -63.99, -64.0, -64.01, -64.5, -70.0, -87.0, -89.0, -104.0, -150.0, -1000.0, -30000.0,
        0.0, 15.0, 90.0, 200.0, 1000.0]


def rows(kind, E, gen):
    T = len(TOPS)
    l = torch.randn(T, E, generator=gen) * {"narrow": 1.0, "wide": 20.0}.get(kind, 3.0)
    l = l - l.amax(1, keepdim=True) + torch.tensor(TOPS)[:, None]
    if kind == "lowest":
        l[:, 1::2] = LOWEST
        l[3] = LOWEST                    # nothing else in the row
    elif kind == "inf":
        l[:, ::3] = -float("inf")
        l[5, 2:] = -float("inf")
    return l


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("kind", ["narrow", "wide", "lowest", "inf"])
@pytest.mark.parametrize("E", [12, 72, 257])
def test_gradients(kind, score, E):
    k = 2 if kind == "inf" and E == 12 else 4
    gen = torch.Generator().manual_seed(E + score)
    l = rows(kind, E, gen)
    T = l.shape[0]
    masked = l == -float("inf")
    ids = torch.topk(l, k, 1).indices.int()
    gw = torch.randn(T, k, generator=gen)
    chosen = l.gather(1, ids.long())
    gw = torch.where(chosen == -float("inf"), 0.0, gw)
    w = torch.where(chosen == -float("inf"), 0.0, ref.routed(l.double(), ids, score).float())

    # -inf would make autograd's products NaN: such entries count as 1e5 below
    # the lowest row, whose probability and gradient are exactly zero
    clean = torch.where(masked, -2e5, l.double()).requires_grad_()
    loss, counts, _, tokens = ref.balance(clean, ids, score, None, COEF)
    want_b = torch.autograd.grad(UP * loss, clean)[0]
    wd, g = w.double(), gw.double()
    d = wd * (g - (g * wd).sum(1, keepdim=True))
    slope = torch.sigmoid(-clean.detach()) if score == 1 else torch.ones_like(clean)
    want_r = torch.zeros(T, E, dtype=torch.float64).scatter_add(1, ids.long(), d) * slope

    # p is off by rel of itself, and where sigmoids fall below the smallest
    # normal number by half of the smallest one over their sum; the exponent's
    # rounding counts with its size
    p = ref.probs(clean.detach(), score)
    finite = torch.where(l < -1e30, 0.0, l.double())
    rel = 2.0 ** -18 + (E + T + 16) * ref.U32 + 4 * ref.U32 * \
        (finite.amax(1, keepdim=True) - finite).abs().amax(1, keepdim=True).clamp(max=200)
    flush = 0.0
    if score == 1:
        total = torch.sigmoid(clean.detach()).sum(1, keepdim=True)
        flush = torch.where(total > 2.0 ** -100, 2.0 ** -149 / total, 0.0)
    gb = UP * COEF * E / k * counts.double() / (T * T)
    size = gb + (gb * p).sum(1, keepdim=True)
    routed = (wd * (g.abs() + (g.abs() * wd).sum(1, keepdim=True)))
    tol_b = 4 * (rel * p + flush) * size + ref.TINY
    tol_r = 4 * rel * torch.zeros(T, E, dtype=torch.float64).scatter_add(1, ids.long(), routed) + ref.TINY

    args = dict(coef=COEF, expert_counts=counts[0].int().view(1, E).cuda(),
                seq_tokens=tokens.int().cuda(), grad_loss=torch.tensor([UP], device="cuda"))
    got_c = api.moe_balance_loss(l.cuda(), None, ids.cuda(), score, COEF)
    assert torch.equal(got_c[1].cpu().long(), counts)
    parts = [(None, None, args, want_b, tol_b), (w.cuda(), gw.cuda(), {}, want_r, tol_r),
             (w.cuda(), gw.cuda(), args, want_b + want_r, tol_b + tol_r)]
    for weights, grads, kw, want, tol in parts:
        got, bias = api.moe_route_backward(l.cuda(), None, ids.cuda(), weights, grads, score,
                                           with_grad_bias=True, **kw)
        off = (got.cpu().double() - want).abs()
        assert (off <= tol).all(), (int((off > tol).sum()), (off > tol).nonzero()[0].tolist(),
                                    float((off / tol).max()))
        assert (got.cpu()[masked] == 0).all()
        bound = tol.sum(0) + (T + 8) * ref.U32 * want.abs().sum(0)
        assert ((bias.cpu().double() - want.sum(0)).abs() <= bound).all()
