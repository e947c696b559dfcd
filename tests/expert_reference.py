"""Plain fp64 forms of the expert product, the combine's and the router's
gradients (CPU torch), and the error bounds their fp32/bf16 results are held to.

U16 is the largest relative error of a rounding to bf16 (half a step), U32 of
one fp32 operation taken at a whole step, so that it also covers sums that cut
instead of rounding.  A sum of n products in fp32 is off by at most
(n + 8) * U32 times the sum of the products' magnitudes, in any order.
"""
import math

import torch

U16 = 2.0 ** -8
U32 = 2.0 ** -23
EXP = 2.0 ** -20      # relative error allowed to the exp/erf of an activation
TINY = 2.0 ** -126    # below it a bf16 or fp32 result may flush
SLOPE = 1.13          # largest slope of silu (1.10) and gelu (1.13)

ACTS = ("none", "silu", "gelu", "swiglu")


def act(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        return g * torch.sigmoid(g) * u
    return z


def segments(counts, offsets, L, C):
    """[begin, end) of every expert's placed rows."""
    out = []
    for e, (c, o) in enumerate(zip(counts, offsets)):
        end = o + c
        if C > 0:
            end = min(end, (e // L) * C + C)
        out.append((o, max(end, o)))
    return out


def matmul(x, w, bias, residual, spans, name, F):
    """y, z and the bounds of their errors, fp64 [rows][..]; NaN where no row is placed."""
    rows, P = x.shape[0], w.shape[1]
    K = x.shape[1]
    y = torch.full((rows, F), float("nan"), dtype=torch.float64)
    z = torch.full((rows, P), float("nan"), dtype=torch.float64)
    ty, tz = torch.zeros_like(y), torch.zeros_like(z)
    for e, (a, b) in enumerate(spans):
        if a == b:
            continue
        ze = x[a:b] @ w[e].T
        dz = x[a:b].abs() @ w[e].abs().T
        if bias is not None:
            ze = ze + bias[e]
            dz = dz + bias[e].abs()
        dz = (K + 8) * U32 * dz
        ye = act(name, ze)
        if name == "swiglu":
            g, u = ze.chunk(2, -1)
            dg, du = dz.chunk(2, -1)
            dy = SLOPE * dg * (u.abs() + du) + act("silu", g).abs() * du + EXP * ye.abs()
        elif name == "none":
            dy = dz
        else:
            dy = SLOPE * dz + EXP * (ye.abs() + ze.abs())
        if residual is not None:
            ye = ye + residual[a:b]
            dy = dy + U32 * ye.abs()
        y[a:b], z[a:b] = ye, ze
        ty[a:b] = dy + U16 * (ye.abs() + dy) + TINY
        tz[a:b] = dz + U16 * (ze.abs() + dz) + TINY
    return y, z, ty, tz


def act_grad(name, z, gy):
    z = z.detach().clone().requires_grad_()
    return torch.autograd.grad((act(name, z) * gy).sum(), z)[0]


def matmul_grad(gy, x, w, pre, spans, name):
    """grad_x, grad_w, grad_b and their bounds: gz enters the products rounded
    to bf16, its sum does not."""
    rows, K = x.shape
    E, P = w.shape[:2]
    gx = torch.full((rows, K), float("nan"), dtype=torch.float64)
    gw, gb = torch.zeros(E, P, K, dtype=torch.float64), torch.zeros(E, P, dtype=torch.float64)
    tx, tw, tb = torch.zeros_like(gx), torch.zeros_like(gw), torch.zeros_like(gb)
    for e, (a, b) in enumerate(spans):
        if a == b:
            continue
        gz = gy[a:b] if name == "none" else act_grad(name, pre[a:b], gy[a:b])
        # the activation's slope in fp32: s (1 + z (1 - s)) and the like
        dgz = 0.0 * gz
        if name != "none":
            scale = gy[a:b].abs() * (1.0 + pre[a:b].abs().amax(1, keepdim=True)) ** 2
            dgz = EXP * (scale.repeat(1, P // scale.shape[1]))
        rz = dgz + U16 * (gz.abs() + dgz) if name != "none" else dgz
        gx[a:b] = gz @ w[e]
        tx[a:b] = (rz + (P + 8) * U32 * (gz.abs() + rz)) @ w[e].abs()
        gw[e] = gz.T @ x[a:b]
        tw[e] = (rz + (b - a + 8) * U32 * (gz.abs() + rz)).T @ x[a:b].abs()
        gb[e] = gz.sum(0)
        tb[e] = (dgz + (b - a + 8) * U32 * gz.abs()).sum(0)
    tx += U16 * (gx.nan_to_num().abs() + tx) + TINY
    tw += U16 * (gw.abs() + tw) + TINY
    return (gx, gw, gb), (tx, tw, tb + TINY)


def widen(codes, scales, rows):
    """fp64 values of e4m3 codes (uint8) with a scale per rows x 128 block."""
    v = codes.view(torch.float8_e4m3fn).float().double()
    s = scales.double().repeat_interleave(128, -1).repeat_interleave(rows, -2)
    return v * s[..., :v.shape[-2], :]


def check(got, want, bound, what, untouched=None):
    """got within bound of want; where want is NaN (a row nobody owns) got must
    still hold the value it was filled with."""
    got = got.double().cpu()
    own = ~want.isnan()
    off = (got - want).abs()
    bad = own & ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(),
                           float(off[bad][0]), float(bound[bad][0]))
    if untouched is not None:
        assert (got[~own] == untouched).all(), what + ": a row of no segment was written"


# ---------------------------------------------------------------------------
# the router
# ---------------------------------------------------------------------------
def probs(l, score):
    if score == 1:
        # sigmoid(l) / sum of them, through logarithms so that nothing vanishes
        return torch.softmax(torch.nn.functional.logsigmoid(l), 1)
    return torch.softmax(l, 1)


def balance(l, ids, score, offsets, coef):
    """(loss, counts [S,E], probs [S,E], tokens [S]) of biased logits l (fp64)."""
    T, E = l.shape
    k = ids.shape[1]
    cuts = [0, T] if offsets is None else [min(max(int(v), 0), T) for v in offsets]
    p = probs(l, score)
    S = len(cuts) - 1
    counts = torch.zeros(S, E, dtype=torch.int64)
    mean = torch.zeros(S, E, dtype=torch.float64)
    tokens = torch.zeros(S, dtype=torch.int64)
    loss = l.new_zeros(())
    for s in range(S):
        keep = [t for t in range(cuts[s], cuts[s + 1])
                if ((ids[t] >= 0) & (ids[t] < E)).any()]
        n = len(keep)
        tokens[s] = n
        if n == 0:
            continue
        flat = ids[keep].flatten().long()
        counts[s] = torch.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
        m = p[keep].sum(0) / n
        mean[s] = m.detach()
        loss = loss + coef / S * (E / (k * n) * counts[s].double() * m).sum()
    return loss, counts, mean, tokens


def routed(l, ids, score):
    """The router's weights of the given slots as a function of the logits:
    normalised over all slots, those with a bad id included through the value
    they would have (their gradient is dropped by the caller)."""
    v = l.gather(1, ids.clamp(0, l.shape[1] - 1).long())
    s = torch.nn.functional.logsigmoid(v) if score == 1 else v
    return torch.softmax(s, 1)
