"""The router's balance loss and the router's gradient against fp64: the
formulas by autograd, central differences, ragged and empty sequences, padding,
extreme logits, repeated ids."""
import pytest
import torch

import expert_reference as ref
from combine_moe_dispatch_amd import api

pytestmark = pytest.mark.gpu

COEF = 0.5


def make(T, E, k, score, bias, offsets, pad, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    l = scale * torch.randn(T, E, generator=gen)
    b = torch.randn(E, generator=gen) if bias else None
    biased = l if b is None else l + b
    ids = torch.topk(biased, k, 1).indices.int()
    if pad and T > 2:
        ids[1::3] = -1
        ids[2::3, 0] = E + 5
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    w = ref.routed(biased.double(), torch.topk(biased, k, 1).indices, score).float()
    gw = torch.randn(T, k, generator=gen)
    gw[(ids < 0) | (ids >= E)] = float("nan")  # must not matter
    if pad and T > 2:
        l[1::3] = float("nan")  # logits of padded tokens must not matter
    return l, b, ids, off, w, gw


def c(t):
    return None if t is None else t.cuda()


def forward(l, b, ids, off, score):
    return api.moe_balance_loss(c(l), c(b), c(ids), score, COEF, c(off))


def reference(l, b, ids, off, score, w, gw, with_balance=True, with_routed=True):
    """fp64 results and bounds: gradients of coef loss and of sum(gw * weights)."""
    E = l.shape[1]
    real = (ids >= 0) & (ids < E)
    clean = torch.where(real.any(1)[:, None], l, 0.0).double().requires_grad_()
    biased = clean if b is None else clean + b.double()
    loss, counts, mean, tokens = ref.balance(biased, ids, score,
                                             None if off is None else off.tolist(), COEF)
    total = clean.sum() * 0.0
    if with_balance:
        total = total + 0.75 * loss
    if with_routed:
        # the weights were normalised over the slots the router chose, so a slot
        # whose id is bad now keeps its share: use the given weights' formula
        s = ref.routed(biased, ids, score)
        lw = biased.gather(1, ids.clamp(0, E - 1).long())
        g = torch.where(real, gw, 0.0).double()
        wd = w.double()
        d = torch.where(real, wd * (g - (g * wd).sum(1, keepdim=True)), 0.0)
        if score == 1:
            d = d * torch.sigmoid(-lw).detach()
        total = total + (d.detach() * lw).sum()
        del s
    grad = torch.autograd.grad(total, clean)[0]
    return float(loss.detach()), counts, mean, tokens, grad


CASES = [
    # T, E, k, bias, offsets, pad
    (1, 1, 1, False, None, False),
    (1, 8, 2, True, None, False),
    (16, 8, 2, False, None, False),
    (7, 64, 5, True, [0, 0, 3, 3, 7, 7], False),
    (130, 65, 8, True, [2, 50, 51, 128], True),
    (300, 256, 8, False, [0, 100, 300], True),
    (90, 384, 8, True, None, True),
    (40, 1024, 32, False, [0, 13, 40], False),
    (1000, 33, 1, True, [0, 1, 2, 500, 501, 777, 900, 1000], True),
    (2500, 129, 4, True, [10, 1030, 1030, 2400], True),
]


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,k,bias,offsets,pad", CASES)
def test_loss_and_gradients(T, E, k, bias, offsets, pad, score):
    l, b, ids, off, w, gw = make(T, E, k, score, bias, offsets, pad, T + E)
    want_loss, want_c, want_p, want_n, want = reference(l, b, ids, off, score, w, gw)
    loss, counts, probs, tokens = forward(l, b, ids, off, score)
    assert torch.equal(counts.cpu().long(), want_c) and torch.equal(tokens.cpu().long(), want_n)
    # p: exp and sums of E terms, relative; then the mean's sum of n terms
    rel = 2.0 ** -18 + (E + T + 16) * ref.U32
    assert ((probs.cpu().double() - want_p).abs() <= rel * want_p + ref.TINY).all()
    assert abs(float(loss) - want_loss) <= (rel + 2 * E * ref.U32) * want_loss + ref.TINY

    gl = torch.tensor([0.75], device="cuda")
    args = dict(coef=COEF, seq_offsets=c(off), expert_counts=counts, seq_tokens=tokens,
                grad_loss=gl)
    got, gb = api.moe_route_backward(c(l), c(b), c(ids), c(w), c(gw), score, with_grad_bias=True,
                                     **args)
    # sums of products of magnitude |g| p and |gw| w cancel: bound by their size
    only_b = reference(l, b, ids, off, score, w, gw, True, False)[4]
    size = magnitude(l, b, ids, off, score, w, gw, want_c, want_n)
    tol = rel * 4 * size + ref.TINY
    assert ((got.cpu().double() - want).abs() <= tol).all()
    bias_tol = tol.sum(0) + (T + 8) * ref.U32 * want.abs().sum(0)
    assert ((gb.cpu().double() - want.sum(0)).abs() <= bias_tol).all()
    # each part alone, and grad_bias left out
    part, none = api.moe_route_backward(c(l), c(b), c(ids), None, None, score, **args)
    assert none is None
    assert ((part.cpu().double() - only_b).abs() <= tol).all()
    only_r = reference(l, b, ids, off, score, w, gw, False, True)[4]
    part, _ = api.moe_route_backward(c(l), c(b), c(ids), c(w), c(gw), score)
    assert ((part.cpu().double() - only_r).abs() <= tol).all()


def magnitude(l, b, ids, off, score, w, gw, counts, tokens):
    """Sizes of the terms that make up each gradient entry."""
    T, E = l.shape
    k = ids.shape[1]
    real = (ids >= 0) & (ids < E)
    p = torch.where(real.any(1)[:, None], ref.probs(
        (torch.where(real.any(1)[:, None], l, 0.0) + (0.0 if b is None else b)).double(), score), 0.0)
    cuts = [0, T] if off is None else off.tolist()
    S = len(cuts) - 1
    g = torch.zeros(T, E, dtype=torch.float64)
    for s in range(S):
        n = max(int(tokens[s]), 1)
        g[cuts[s]:cuts[s + 1]] = 0.75 * COEF / S * E / k * counts[s].double() / (n * n)
    size = p * (g + (g * p).sum(1, keepdim=True))
    a = torch.where(real, gw.abs(), 0.0).double()
    r = torch.where(real, w.double() * (a + (a * w.double()).sum(1, keepdim=True)), 0.0)
    return size.scatter_add(1, torch.where(real, ids, 0).long(), r)


@pytest.mark.parametrize("score", [0, 1])
def test_differences(score):
    """Gradients against central differences of the fp64 loss."""
    T, E, k = 12, 10, 3
    l, b, ids, off, w, gw = make(T, E, k, score, True, [0, 5, 12], False, 4)
    _, counts, _, tokens = forward(l, b, ids, off, score)
    got, gb = api.moe_route_backward(c(l), c(b), c(ids), c(w), c(gw), score, coef=COEF,
                                     seq_offsets=c(off), expert_counts=counts, seq_tokens=tokens,
                                     with_grad_bias=True)

    def value(lg, bs):
        biased = lg + bs
        return float(ref.balance(biased, ids, score, off.tolist(), COEF)[0] +
                     (gw.double() * ref.routed(biased, ids, score)).sum())

    gen = torch.Generator().manual_seed(1)
    h = 1e-5
    for _ in range(8):
        dl = torch.randn(T, E, generator=gen, dtype=torch.float64)
        db = torch.randn(E, generator=gen, dtype=torch.float64)
        up = value(l.double() + h * dl, b.double() + h * db)
        down = value(l.double() - h * dl, b.double() - h * db)
        want = (up - down) / (2 * h)
        have = float((got.cpu().double() * dl).sum() + (gb.cpu().double() * db).sum())
        # fp32 results (2^-18 of each entry's size) and the differences' own h^2
        assert abs(want - have) <= 2.0 ** -14 * float((got.cpu().abs() * dl.abs()).sum()) + 1e-7


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("kind", ["lowest", "very_low", "large", "inf"])
def test_extreme_logits(score, kind):
    """The type's lowest value or -inf as a mask, sigmoids that vanish, wide logits."""
    T, E, k = 20, 40, 4
    gen = torch.Generator().manual_seed(2)
    l = torch.randn(T, E, generator=gen)
    if kind == "lowest":
        l[:, ::2] = torch.finfo(torch.float32).min
    elif kind == "inf":
        l[:, 1::2] = -float("inf")
    elif kind == "very_low":
        l -= 150.0
    else:
        l *= 60.0
    ids = torch.topk(l, k, 1).indices.int()
    loss, counts, probs, tokens = forward(l, None, ids, None, score)
    want_loss, want_c, want_p, _ = ref.balance(l.double(), ids, score, None, COEF)
    rel = 2.0 ** -18 + (E + T) * ref.U32 + float(l[l > -1e30].abs().max()) * ref.U32 * 2
    assert ((probs.cpu().double() - want_p).abs() <= rel * want_p + ref.TINY).all()
    assert abs(float(loss) - float(want_loss)) <= rel * 2 * float(want_loss)
    got, _ = api.moe_route_backward(c(l), None, c(ids), None, None, score, coef=COEF,
                                    expert_counts=counts, seq_tokens=tokens)
    assert got.isfinite().all()


def test_no_tokens_and_all_padded():
    for T in (0, 9):
        l = torch.randn(T, 8)
        ids = torch.full((T, 2), -1, dtype=torch.int32)
        off = torch.tensor([0, 4, 9], dtype=torch.int32)
        loss, counts, probs, tokens = forward(l, None, ids, off, 1)
        assert float(loss) == 0 and (counts == 0).all() and (probs == 0).all() and (tokens == 0).all()
        got, gb = api.moe_route_backward(c(l), None, c(ids), None, None, 1, coef=COEF,
                                         seq_offsets=c(off), expert_counts=counts,
                                         seq_tokens=tokens, with_grad_bias=True)
        assert (got == 0).all() and (gb == 0).all() and got.shape == (T, 8)


def test_repeated_ids_add_up():
    l = torch.randn(5, 6)
    ids = torch.tensor([[1, 1, 2]] * 5, dtype=torch.int32)
    w = torch.tensor([[0.5, 0.2, 0.3]] * 5)
    gw = torch.randn(5, 3)
    got, _ = api.moe_route_backward(c(l), None, c(ids), c(w), c(gw), 0)
    d = w.double() * (gw.double() - (gw.double() * w.double()).sum(1, keepdim=True))
    want = torch.zeros(5, 6, dtype=torch.float64)
    want[:, 1] = d[:, 0] + d[:, 1]
    want[:, 2] = d[:, 2]
    assert ((got.cpu().double() - want).abs() <= 16 * ref.U32 * gw.abs().amax(1, keepdim=True)).all()
    _, counts, _, _ = forward(l, None, ids, None, 0)
    assert counts.cpu().tolist() == [[0, 10, 5, 0, 0, 0]]


def test_offsets_outside_the_batch_are_cut():
    l = torch.randn(10, 8)
    ids = torch.topk(l, 2, 1).indices.int()
    a = forward(l, None, ids, torch.tensor([-4, 6, 40], dtype=torch.int32), 1)
    b = forward(l, None, ids, torch.tensor([0, 6, 10], dtype=torch.int32), 1)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_uniform_routing_gives_coef():
    T, E, k = 64, 16, 4
    l = torch.zeros(T, E)
    ids = torch.stack([(torch.arange(k) + t * k) % E for t in range(T)]).int()
    loss, _, _, _ = forward(l, None, ids, None, 0)
    assert abs(float(loss) - COEF) <= 1e-5 * COEF


def test_large_batch_is_deterministic():
    l, b, ids, off, w, gw = make(20000, 256, 8, 1, True, [0, 7000, 7001, 20000], True, 8)
    first = forward(l, b, ids, off, 1)
    again = forward(l, b, ids, off, 1)
    for x, y in zip(first, again):
        assert torch.equal(x, y)
    kw = dict(coef=COEF, seq_offsets=c(off), expert_counts=first[1], seq_tokens=first[3],
              with_grad_bias=True)
    a = api.moe_route_backward(c(l), c(b), c(ids), c(w), c(gw), 1, **kw)
    d = api.moe_route_backward(c(l), c(b), c(ids), c(w), c(gw), 1, **kw)
    assert torch.equal(a[0], d[0]) and torch.equal(a[1], d[1])
    assert torch.equal(first[3].cpu().long(),
                       ref.balance(torch.zeros(20000, 256, dtype=torch.float64), ids, 1,
                                   off.tolist(), COEF)[3])


@pytest.mark.parametrize("E", [64, 256, 384, 1024])
def test_misaligned_arrays(E):
    """Logits, bias, counts and outputs four bytes past a 16-byte boundary: the same values."""
    T, k = 200, 3
    l, b, ids, off, w, gw = make(T, E, k, 1, True, [0, 90, 200], False, 3)

    def odd(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:].copy_(t.flatten())
        return flat[1:].view(t.shape)

    want = api.moe_balance_loss(c(l), c(b), c(ids), 1, COEF, c(off))
    got = api.moe_balance_loss(odd(l), odd(b), odd(ids), 1, COEF, odd(off))
    # the order of a row's sum differs, so fp32 sums of E terms and their mean
    assert torch.equal(got[1], want[1]) and torch.equal(got[3], want[3])
    rel = (2 * E + T) * ref.U32
    assert ((got[2] - want[2]).abs() <= rel * want[2]).all()
    kw = dict(coef=COEF, expert_counts=want[1], seq_tokens=want[3])
    a, _ = api.moe_route_backward(c(l), c(b), c(ids), c(w), c(gw), 1, seq_offsets=c(off), **kw)
    out = odd(torch.zeros(T, E))
    d, _ = api.moe_route_backward(odd(l), odd(b), c(ids), odd(w), odd(gw), 1, seq_offsets=c(off),
                                  grad_logits=out, **kw)
    size = magnitude(l, b, ids, off, 1, w, gw, want[1].cpu(), want[3].cpu())
    assert d is out
    assert ((a - d).abs().cpu().double() <= 2 * rel * size / 0.75 + ref.TINY).all()


@pytest.mark.parametrize("T,first,run", [(30, 11, 100000), (500, 16, 300000), (500, 250, 7), (0, 0, 50)])
def test_long_runs_of_empty_sequences(T, first, run):
    """Empty sequences between two others, more than there are tokens: the same
    values as without them."""
    l, b, ids, _, w, gw = make(T, 40, 3, 1, True, None, False, 4)
    short = torch.tensor([0, first, T], dtype=torch.int32)
    long = torch.tensor([0] + [first] * (run + 1) + [T], dtype=torch.int32)
    S, at = run + 2, [0, run + 1]
    loss, counts, probs, tokens = forward(l, b, ids, short, 1)
    got = forward(l, b, ids, long, 1)
    assert torch.equal(got[1][at], counts) and torch.equal(got[3][at], tokens)
    # the same sums over at most 500 tokens, perhaps in another order
    bound = 1024 * ref.U32
    assert ((got[2][at] - probs).abs() <= bound * probs).all()
    for t in got[1:]:
        assert (t[1:-1] == 0).all()
    assert abs(float(got[0]) * S - 2 * float(loss)) <= 2 * bound * 2 * float(loss)
    kw = dict(expert_counts=counts, seq_tokens=tokens)
    want, _ = api.moe_route_backward(c(l), c(b), c(ids), c(w), c(gw), 1, coef=COEF,
                                     seq_offsets=c(short), **kw)
    kw = dict(expert_counts=got[1], seq_tokens=got[3])
    grad, _ = api.moe_route_backward(c(l), c(b), c(ids), c(w), c(gw), 1, coef=COEF * S / 2,
                                     seq_offsets=c(long), **kw)
    # the factor coef / S is rounded in another place: a few roundings of each part,
    # which are at most the balance part (E/k coef / n) and the routed one in size
    size = 2 * 40 / 3 * COEF / max(min(first, T - first), 1) + gw.abs().amax(1, keepdim=True) \
        if T else torch.zeros(0, 1)
    assert ((grad - want).abs().cpu() <= 16 * ref.U32 * size).all()


@pytest.mark.parametrize("T", [1, 64, 65])
@pytest.mark.parametrize("S", [3, 4, 5, 64, 200])
def test_few_tokens_in_many_sequences(T, S):
    offsets = [min(i * T // S, T) for i in range(S)] + [T]
    l, b, ids, off, w, gw = make(T, 72, 5, 0, False, offsets, True, T + S)
    loss, counts, probs, tokens = forward(l, b, ids, off, 0)
    want, cnt, mean, n, _ = reference(l, b, ids, off, 0, w, gw)
    assert torch.equal(counts.cpu().long(), cnt.long()) and torch.equal(tokens.cpu().long(), n.long())
    # softmax entries: exp of a difference (its rounding, |l - top| <= 16 half ulps, and
    # the function's few ulps), sums of 72 entries and of T tokens
    assert ((probs.cpu().double() - mean).abs() <= (16 + 8 + 72 + T + 8) * ref.U32 * mean + 1e-30).all()
    assert abs(float(loss) - want) <= (16 + 8 + 72 + T + S + 16) * ref.U32 * want


def test_one_expert_in_every_slot_is_deterministic():
    """32 slots with the same id: their gradients add up in the slots' order."""
    T, E, k = 300, 64, 32
    gen = torch.Generator().manual_seed(2)
    l = torch.randn(T, E, generator=gen)
    ids = torch.full((T, k), 7, dtype=torch.int32)
    w = torch.rand(T, k, generator=gen)
    gw = torch.randn(T, k, generator=gen) * 10 ** (4 * torch.rand(T, k, generator=gen))
    got = [api.moe_route_backward(c(l), None, c(ids), c(w), c(gw), 0)[0] for _ in range(4)]
    for g in got[1:]:
        assert torch.equal(g, got[0])
    d = w.double() * (gw.double() - (gw.double() * w.double()).sum(1, keepdim=True))
    # the inner sum and the outer one each have 32 terms (5 + 32 roundings of partial sums)
    inner = (gw.double() * w.double()).abs().sum(1)
    bound = 40 * ref.U32 * (w.double() * (gw.double().abs() + inner[:, None])).sum(1) * 2
    assert ((got[0][:, 7].cpu().double() - d.sum(1)).abs() <= bound).all()
    assert (got[0][:, :7] == 0).all() and (got[0][:, 8:] == 0).all()
