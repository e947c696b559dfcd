"""Plain fp64 forms of the expert layer in 8 bits (CPU torch) and the bounds that
its results are held to.  Roundings are counted as in expert_reference; an e4m3
rounding is half a step, 2^-4 of the value or 2^-10 of the block's scale.

A rounding to 8 bits can land on another code only where the value may lie on the
other side of a border: `quantize` takes the bounds of the values' errors and gives
how far the rounded ones can be from the reference's.
"""
import numpy as np
import torch

import expert_reference as ref
from expert_reference import EXP, SLOPE, TINY, U16, U32

CUT = 8 * 2.0 ** -13   # of the largest of 8 neighbouring products (test_gpu_fp8_sums)
STEPS = 8              # fp32 operations allowed to a norm's value besides its sums


def e4m3(q):
    """Nearest e4m3 values, ties to even, magnitudes cut at 448."""
    exponent = torch.frexp(q).exponent - 1
    step = torch.ldexp(torch.ones_like(q), exponent.clamp(min=-6) - 3)
    return (torch.round(q / step) * step).clamp(-448.0, 448.0)


def codes_of(v):
    """Codes' values and scales of fp32 rows (exactly as defined: fp32 divisions)."""
    a = v.float().numpy().reshape(*v.shape[:-1], -1, 128)
    with np.errstate(all="ignore"):
        s = np.abs(a).max(-1) / np.float32(448)
        q = np.where(s[..., None] > 0, a / s[..., None], np.float32(0))
    codes = e4m3(torch.from_numpy(q.astype(np.float64)))
    return codes.flatten(-2), torch.from_numpy(s)


def quantize(v, dv):
    """Rounded values of v, known to dv, in blocks of 128 columns, and their slack."""
    v, dv = v.unflatten(-1, (-1, 128)), dv.unflatten(-1, (-1, 128))
    s = (v.abs().amax(-1, keepdim=True) / 448.0).clamp(min=2.0 ** -149)
    ds = dv.amax(-1, keepdim=True) / 448.0 + 2.0 ** -23 * s
    q = v / s
    dq = dv / s + q.abs() * (ds / s + 2.0 ** -23)
    mid, lo, hi = e4m3(q), e4m3(q - dq), e4m3(q + dq)
    slack = torch.maximum(hi - mid, mid - lo) * (s + ds) + mid.abs() * ds
    return (mid * s).flatten(-2), slack.flatten(-2)


def product(a, da, w):
    """a w^T in 8 bits and its bound: a is known to da; the matrix instruction's cut,
    and fp32 sums."""
    K = a.shape[1]
    largest = torch.zeros(a.shape[0], w.shape[0], dtype=torch.float64)
    for g in range(0, K, 8):
        p = a[:, None, g:g + 8].abs() * w[None, :, g:g + 8].abs()
        largest += p.amax(2)
    magnitude = (a.abs() + da) @ w.abs().T
    z = a @ w.T
    return z, da @ w.abs().T + CUT * largest + (K / 8 + 3 * K / 128 + 8) * U32 * magnitude


def gated(z, dz):
    g, u = z.chunk(2, -1)
    dg, du = dz.chunk(2, -1)
    h = ref.act("swiglu", z)
    return h, SLOPE * dg * (u.abs() + du) + ref.act("silu", g).abs() * du + EXP * h.abs()


def rounded16(v, dv):
    return dv + U16 * (v.abs() + dv) + TINY


def forward(x, up, down, residual):
    """One expert's y and z with their bounds."""
    z, dz = product(x, torch.zeros_like(x), up)
    hq, slack = quantize(*gated(z, dz))
    y, dy = product(hq, slack, down)
    if residual is not None:
        y = y + residual
        dy = dy + U32 * y.abs()
    return (y, rounded16(y, dy)), (z, rounded16(z, dz))


def backward(gy, x, up, down, pre):
    """One expert's gradients of rows and weights with their bounds."""
    codes, scales = codes_of(gy.float())
    gq = (codes.unflatten(-1, (-1, 128)) * scales.double()[..., None]).flatten(-2)
    gh, dgh = product(gq, torch.zeros_like(gq), down.T.contiguous())
    g, u = pre.chunk(2, -1)
    s = torch.sigmoid(g)
    slope_g, slope_u = u * s * (1 + g * (1 - s)), g * s
    gz = torch.cat([gh * slope_g, gh * slope_u], 1)
    # the slope in fp32: products of s, 1 - s, g and u, each a few steps off
    dgz = torch.cat([dgh * slope_g.abs() + (gh.abs() + dgh) * EXP * u.abs() * s * (1 + g.abs()),
                     dgh * slope_u.abs() + (gh.abs() + dgh) * EXP * slope_u.abs()], 1)
    zq, slack = quantize(gz, dgz)
    gx, dgx = product(zq, slack, up.T.contiguous())
    n = gy.shape[0]
    def summed(a, da, b, db):
        v = a.T @ b
        d = da.T @ (b.abs() + db) + a.abs().T @ db + (n + 8) * U32 * (a.abs() + da).T @ (b.abs() + db)
        return v, rounded16(v, d)
    h = g * s * u
    gup = summed(gz, rounded16(gz, dgz), x, U16 * x.abs() + TINY)
    gdown = summed(gy, torch.zeros_like(gy), h, rounded16(h, EXP * h.abs()))
    return (gx, rounded16(gx, dgx)), gup, gdown


def norm(t, w, eps):
    """v = t / rms * w and 1 / rms, with the bounds of their errors."""
    H = t.shape[1]
    r = ((t * t).mean(1, keepdim=True) + eps).rsqrt()
    dr = ((H + 8) / 2 * U32 + STEPS * U32) * r
    v = t * r * w
    return v, v.abs() * (dr / r + 4 * U32), r.flatten(), dr.flatten()


def norm_grad(gy, t, w, r, carried):
    H = t.shape[1]
    r = r[:, None]
    n, a = t * r, gy * w
    mean = (a * n).mean(1, keepdim=True)
    gx = r * (a - n * mean)
    dmean = (H + 8) * U32 * (a * n).abs().mean(1, keepdim=True)
    dgx = r * (STEPS * U32 * (a.abs() + (n * mean).abs()) + n.abs() * dmean)
    if carried is not None:
        gx = gx + carried
        dgx = dgx + U32 * (gx.abs() + carried.abs())
    gw = (gy * n).sum(0)
    return (gx, rounded16(gx, dgx)), (gw, (t.shape[0] + 8) * U32 * (gy * n).abs().sum(0) + TINY)
