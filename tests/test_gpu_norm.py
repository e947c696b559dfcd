"""The RMS norm, its gradient and 8-bit weights against plain fp64 forms: one row to
many, every thread layout, odd sizes, optional outputs, in-place use, masks of NaN
and infinities, empty rows and blocks."""
import numpy as np
import pytest
import torch

import ffn_reference as plain
from combine_moe_dispatch_amd import api
from expert_reference import TINY, U16

pytestmark = pytest.mark.gpu

EPS = 1e-6
FILL = -7.0


def rows(T, H, seed, loud=True):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=gen)
    if loud:
        x = x * (1 + 20.0 * (torch.rand(H, generator=gen) < 0.01))
    return x.bfloat16()


def norm_weight(H, seed):
    return 1.0 + 0.2 * torch.randn(H, generator=torch.Generator().manual_seed(seed + 100))


def out(T, H, dtype=torch.bfloat16):
    fill = 0x55 if dtype == torch.uint8 else FILL
    return torch.full((T + 1, H), fill, dtype=dtype, device="cuda")  # one canary row


def check(got, want, bound, what):
    off = (got.double().cpu() - want).abs()
    assert (off <= bound).all(), (what, float((off - bound).max()))


def check_codes(codes, scales, v, dv):
    """Codes within the two that the value's error allows, scales within theirs."""
    got = codes.cpu().view(torch.float8_e4m3fn).double()
    value, slack = plain.quantize(v, dv)
    s = scales.double().cpu()
    check((got.unflatten(1, (-1, 128)) * s[..., None]).flatten(1), value, slack + TINY, "8-bit rows")
    want = v.abs().unflatten(1, (-1, 128)).amax(2) / 448
    ds = dv.unflatten(1, (-1, 128)).amax(2) / 448
    check(s, want, ds + 2.0 ** -23 * want + TINY, "scales")


def run(T, H, residual=True, codes=True, y=True, total=True, inv=True, seed=0):
    x, w = rows(T, H, seed), norm_weight(H, seed)
    res = rows(T, H, seed + 1, loud=False) if residual else None
    t, yy, inv_ = (out(T, H) if total else None), (out(T, H) if y else None), None
    c, s = (out(T, H, torch.uint8), out(T, H // 128, torch.float32)) if codes else (None, None)
    if inv:
        inv_ = torch.full((T + 1,), FILL, device="cuda")
    api.moe_rms_norm(x.cuda(), None if res is None else res.cuda(), w.cuda(), EPS, t, yy, c, s, inv_)
    want_t = x if res is None else (x.float() + res.float()).bfloat16()
    v, dv, r, dr = plain.norm(want_t.double(), w.double(), EPS)
    if total:
        assert torch.equal(t[:T].cpu(), want_t) and (t[T] == FILL).all()
    if y:
        check(yy[:T], v, plain.rounded16(v, dv), "y")
        assert (yy[T] == FILL).all()
    if codes:
        check_codes(c[:T], s[:T], v, dv)
        assert (c[T] == 0x55).all() and (s[T] == FILL).all()
    if inv:
        check(inv_[:T], r, dr, "1 / rms")
        assert inv_[T] == FILL


@pytest.mark.parametrize("T,H", [(1, 128), (1, 7168), (2, 8192), (3, 8320), (255, 384), (256, 2048),
                                 (257, 2176), (300, 4096), (257, 4224), (700, 128), (1500, 256),
                                 (270, 8192), (5, 16384), (3, 16512), (2, 32768), (2, 40960),
                                 (1, 65536)])
def test_norm(T, H):
    run(T, H, seed=T + H)


@pytest.mark.parametrize("T,H", [(1, 8), (7, 72), (300, 1432), (257, 2056), (4, 20008), (2100, 8)])
def test_norm_of_odd_rows(T, H):
    run(T, H, codes=False, seed=T)
    run(T, H, codes=False, residual=False, seed=T)


@pytest.mark.parametrize("kw", [dict(residual=False), dict(y=False), dict(codes=False),
                                dict(total=False), dict(inv=False),
                                dict(residual=False, total=False, y=False, inv=False),
                                dict(total=False, y=False, codes=False)])
def test_norm_with_some_outputs(kw):
    run(40, 640, **kw)
    run(400, 640, **kw)


@pytest.mark.parametrize("T", [3, 2500])
def test_norm_in_place(T):
    """total over the residual and y over x; rows of several passes of a block."""
    H = 512
    x, res, w = rows(T, H, 5).cuda(), rows(T, H, 6).cuda(), norm_weight(H, 5).cuda()
    t, y = torch.empty_like(x), torch.empty_like(x)
    api.moe_rms_norm(x, res, w, EPS, t, y)
    api.moe_rms_norm(x, res, w, EPS, res, x)
    assert torch.equal(res, t) and torch.equal(x, y)


def test_norm_of_special_rows():
    """Zeros, a NaN, an infinity, the largest and the smallest values, a block of zeros."""
    H = 384
    x = rows(8, H, 9)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 130] = float("inf")
    x[3] = 1e15
    x[4] = 1e-30
    x[5, 128:256] = 0
    w = torch.ones(H)
    w[256:] = 0                     # a block that the weights clear
    xg = x.cuda()
    y, c = torch.empty_like(xg), torch.empty(8, H, dtype=torch.uint8, device="cuda")
    s = torch.empty(8, H // 128, device="cuda")
    api.moe_rms_norm(xg, None, w.cuda(), EPS, None, y, c, s)
    y, c, s = y.cpu(), c.cpu().view(torch.float8_e4m3fn).float(), s.cpu()
    assert (y[0] == 0).all() and (c[0] == 0).all() and (s[0] == 0).all()
    assert y[1].isnan().all() and s[1].isnan().all() and c[1].isnan().all()
    assert y[2, 130].isnan() and s[2, 1].isnan() and c[2, 128:256].isnan().all()
    fine = [3, 4, 5, 6, 7]
    v, dv, _, _ = plain.norm(x[fine].double(), w.double(), EPS)
    check(y[fine], v, plain.rounded16(v, dv), "y")
    assert (c[fine][:, 256:] == 0).all() and (s[fine, 2] == 0).all() and (c[5, 128:256] == 0).all()
    assert (c[3, :256] == 448).all()


def test_codes_of_infinite_values():
    """A norm cannot give infinities of its own; a weight can."""
    H = 128
    w = torch.ones(H)
    w[3] = float("inf")
    x = torch.ones(1, H, dtype=torch.bfloat16, device="cuda")
    c, s = torch.empty(1, H, dtype=torch.uint8, device="cuda"), torch.empty(1, 1, device="cuda")
    api.moe_rms_norm(x, None, w.cuda(), EPS, None, None, c, s)
    c = c.cpu().view(torch.float8_e4m3fn).float()[0]
    assert s.item() == float("inf") and c[3].isnan()
    assert (c[torch.arange(H) != 3] == 0).all()


def grads(T, H, carried=True, gx=True, gw=True, seed=0):
    t, w = rows(T, H, seed), norm_weight(H, seed)
    gen = torch.Generator().manual_seed(seed + 7)
    gy = (0.01 * torch.randn(T, H, generator=gen)).bfloat16()
    c = (0.01 * torch.randn(T, H, generator=gen)).bfloat16() if carried else None
    r = (t.double().square().mean(1) + EPS).rsqrt().float()
    x_out = out(T, H) if gx else None
    w_out = torch.full((H + 8,), FILL, device="cuda") if gw else None
    ws = api.alloc_rms_norm_workspace(T, H, "cuda")
    if ws is not None:
        ws.fill_(0xFF)
    api.moe_rms_norm_backward(gy.cuda(), t.cuda(), w.cuda(), r.cuda(),
                              None if c is None else c.cuda(), x_out, w_out, ws)
    want_x, want_w = plain.norm_grad(gy.double(), t.double(), w.double(), r.double(),
                                     None if c is None else c.double())
    if gx:
        check(x_out[:T], *want_x, "grad_x")
        assert (x_out[T] == FILL).all()
    if gw:
        check(w_out[:H], *want_w, "grad_weight")
        assert (w_out[H:] == FILL).all()


@pytest.mark.parametrize("T,H", [(1, 8), (1, 7168), (2, 72), (9, 8200), (255, 1432), (256, 2048),
                                 (257, 2056), (513, 264), (600, 4096), (300, 8192), (2100, 136),
                                 (3, 16384), (5, 16392), (2, 40960), (1, 65536)])
def test_norm_gradient(T, H):
    grads(T, H, seed=T + H)


@pytest.mark.parametrize("kw", [dict(carried=False), dict(gx=False), dict(gw=False)])
def test_norm_gradient_of_some(kw):
    grads(33, 640, **kw)
    grads(900, 640, **kw)


@pytest.mark.parametrize("T,H,kw", [(150, 16392, {}), (65, 40960, dict(carried=False)), (64, 65536, {}),
                                    (70, 32776, dict(gx=False)), (70, 16392, dict(gw=False)),
                                    (1, 20000, dict(gx=False))])
def test_norm_gradient_of_wide_rows(T, H, kw):
    grads(T, H, seed=T, **kw)


@pytest.mark.parametrize("T,H", [(0, 32768), (90, 32768)])
def test_norm_gradient_of_wide_rows_in_place(T, H):
    t, w = rows(T, H, 3).cuda(), norm_weight(H, 3).cuda()
    gy = rows(T, H, 4).cuda()
    r = (t.double().square().mean(1) + EPS).rsqrt().float()
    gx, gw, again = torch.empty_like(t), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    api.moe_rms_norm_backward(gy, t, w, r, None, gx, gw)
    api.moe_rms_norm_backward(gy, t, w, r, None, gy, again)
    assert torch.equal(gy, gx) and torch.equal(again, gw)
    assert T > 0 or (gw == 0).all()


def test_norm_gradient_without_rows():
    w = torch.ones(64, device="cuda")
    gw = torch.full((64,), FILL, device="cuda")
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    api.moe_rms_norm_backward(none, none, w, w[:0], None, none, gw)
    assert (gw == 0).all()


def test_norm_gradient_in_place_and_repeatable():
    T, H = 1500, 1024
    t, w = rows(T, H, 3).cuda(), norm_weight(H, 3).cuda()
    gy, c = rows(T, H, 4).cuda(), rows(T, H, 5).cuda()
    r = (t.double().square().mean(1) + EPS).rsqrt().float()
    gx, gw = torch.empty_like(t), torch.empty(H, device="cuda")
    api.moe_rms_norm_backward(gy, t, w, r, c, gx, gw)
    for over in (gy.clone(), c.clone()):
        again = torch.empty_like(gw)
        same = over.equal(gy)
        api.moe_rms_norm_backward(over if same else gy, t, w, r, c if same else over, over, again)
        assert torch.equal(over, gx) and torch.equal(again, gw)


def test_norm_gradient_against_differences():
    """The library's own forward sums, read through a linear loss: its rows are
    rounded to bf16, so the steps are wide and the tolerance counts those roundings."""
    T, H = 4, 64
    gen = torch.Generator().manual_seed(2)
    t = torch.randn(T, H, generator=gen).bfloat16()
    gy = torch.randn(T, H, generator=gen).bfloat16()
    w = norm_weight(H, 2)
    r = torch.empty(T, device="cuda")
    api.moe_rms_norm(t.cuda(), None, w.cuda(), EPS, None, None, None, None, r)
    gx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    api.moe_rms_norm_backward(gy.cuda(), t.cuda(), w.cuda(), r, None, gx, None)
    d = torch.randn(T, H, generator=gen)
    d = d / d.norm(dim=1, keepdim=True)
    step = 0.5  # a change of 2^-4 of a row: the third difference is some 2^-8 of the first

    def loss(x):
        y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        api.moe_rms_norm(x.cuda(), None, w.cuda(), EPS, None, y)
        return (y.double().cpu() * gy.double()).sum(1)

    hi, lo = (t.float() + step * d).bfloat16(), (t.float() - step * d).bfloat16()
    got = loss(hi) - loss(lo)
    want = (gx.double().cpu() * (hi.double() - lo.double())).sum(1)
    # both losses round each of H values to half a bf16 step; gx as well; and the
    # cubic term, |d|^2 / H of the first (rms is 1 here)
    v = plain.norm(t.double(), w.double(), EPS)[0].abs()
    bound = 2 * U16 * (1.5 * v * gy.double().abs()).sum(1) + \
        U16 * (gx.double().cpu() * (hi.double() - lo.double())).abs().sum(1) + \
        step ** 2 / H * 4 * gy.double().norm(dim=1) * 2 * step
    assert ((got - want).abs() <= bound).all()
    assert (want.abs() > bound).any()   # the check says something


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,P,K", [(1, 128, 128), (3, 384, 128), (2, 128, 640), (5, 256, 1280)])
def test_weights(E, P, K, dtype):
    """Bit for bit the definition's fp32 divisions."""
    gen = torch.Generator().manual_seed(P + K)
    w = torch.randn(E, P, K, generator=gen)
    w[0, :128, :128] = 0
    w[-1, -1, -1] = 77.0                         # one outlier rules its block
    w[-1, -128:, :128] *= 1e-37                  # a scale below the ordinary range
    w[E // 2, :128, -128:] *= 1e30
    w = w.to(dtype)
    codes = torch.full((E * P * K + 8,), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((E * P * K // 16384 + 1,), FILL, device="cuda")
    api.moe_quantize_weight(w.cuda(), codes, scales)
    b = w.float().numpy().reshape(E, P // 128, 128, K // 128, 128)
    s = np.abs(b).max((2, 4)) / np.float32(448)
    with np.errstate(all="ignore"):
        q = np.where(s[:, :, None, :, None] > 0, b / s[:, :, None, :, None], np.float32(0))
    want = plain.e4m3(torch.from_numpy(q.astype(np.float64))).view(E, P, K)
    assert np.array_equal(scales[:-1].cpu().numpy().reshape(s.shape), s) and scales[-1] == FILL
    got = codes[:-8].cpu().view(torch.float8_e4m3fn).double().view(E, P, K)
    assert torch.equal(got, want)
    assert (codes[-8:] == 0x55).all()


@pytest.mark.parametrize("power", [-149, -148, -140, -126, -81, -80, 79, 80, 81, 100, 117])
def test_weights_of_far_scales(power):
    """Largest magnitudes from one smallest fp32 step to near the largest fp32 value,
    where a scale is coarse or nothing, bit for bit."""
    gen = torch.Generator().manual_seed(power + 200)
    w = torch.randint(-600, 601, (128, 128), generator=gen).double() * 2.0 ** power
    w[5, 7] = 600 * 2.0 ** power
    w = w.float()
    codes, scales = torch.empty(128, 128, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")
    api.moe_quantize_weight(w.cuda(), codes, scales)
    b = w.numpy()
    s = np.abs(b).max() / np.float32(448)
    q = b / s if s > 0 else np.zeros_like(b)
    assert scales.item() == s
    assert torch.equal(codes.cpu().view(torch.float8_e4m3fn).double(),
                       plain.e4m3(torch.from_numpy(q.astype(np.float64))))


def test_weights_with_a_nan():
    w = torch.ones(128, 256)
    w[7, 200] = float("nan")
    w[9, 3] = float("-inf")
    codes, scales = torch.empty(128, 256, dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
    api.moe_quantize_weight(w.cuda(), codes, scales)
    got = codes.cpu().view(torch.float8_e4m3fn).float()
    assert scales[1].isnan() and got[:, 128:].isnan().all()
    assert scales[0] == float("inf") and got[9, 3].isnan()
    got[9, 3] = 0
    assert (got[:, :128] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_signs_of_zeros(dtype):
    """A -0 beside other values keeps its sign, as the division and its rounding would;
    a block of zeros has codes of 0."""
    w = torch.randn(128, 384, generator=torch.Generator().manual_seed(3)).to(dtype)
    w[::3] = -0.0
    w[1::3] = 0.0
    w[:, 128:256] = -0.0
    w[2, 256] = 1e9              # small ones round to zero
    codes, scales = torch.empty(128, 384, dtype=torch.uint8, device="cuda"), torch.empty(3, device="cuda")
    api.moe_quantize_weight(w.cuda(), codes, scales)
    blocks = w.float().numpy().reshape(128, 3, 128)
    s = np.abs(blocks).max((0, 2)) / np.float32(448)
    with np.errstate(all="ignore"):
        q = np.where(s[None, :, None] > 0, blocks / s[None, :, None], np.float32(0))
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).view(128, 384)
    assert torch.equal(codes.cpu(), want) and np.array_equal(scales.cpu().numpy(), s)
    rows = w.bfloat16()
    c, s = torch.empty(128, 384, dtype=torch.uint8, device="cuda"), torch.empty(128, 3, device="cuda")
    api.moe_rms_norm(rows.cuda(), None, torch.ones(384, device="cuda"), EPS, None, None, c, s)
    zeros = (rows == 0) & (s.cpu() > 0).repeat_interleave(128, 1)
    assert torch.equal(c.cpu()[zeros] == 0x80, rows[zeros].signbit())
    assert (c.cpu()[(s.cpu() == 0).repeat_interleave(128, 1)] == 0).all()


def test_refusals_on_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        api.moe_rms_norm(x.t().contiguous().t(), None, w, EPS, None, x)
    with pytest.raises(ValueError, match="weight holds"):
        api.moe_rms_norm(x, None, w[:8], EPS, None, x)
    with pytest.raises(TypeError, match="weight must be"):
        api.moe_rms_norm(x, None, w.bfloat16(), EPS, None, x)
    with pytest.raises(ValueError, match="scales holds"):
        api.moe_rms_norm(x, None, w, EPS, None, None, x.view(torch.uint8), w[:1])
    with pytest.raises(api.MoeError, match="INVALID"):
        api.moe_rms_norm(x, None, w, EPS, x, x)
    with pytest.raises(TypeError, match="weight must be"):
        api.moe_quantize_weight(x.half(), x.view(torch.uint8), w)
    with pytest.raises(api.MoeError):                    # 4 rows are no block
        api.moe_quantize_weight(x, x.view(torch.uint8), w)


def test_rows_past_2_31_elements():
    """Offsets that pass 32 bits."""
    T, H = 300001, 7168
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(0)
    at = [0, 149797, 149798, 299593, 300000]
    x[at] = torch.randn(5, H, generator=gen).bfloat16().cuda()
    w = norm_weight(H, 0)
    y, c = torch.empty_like(x), torch.empty(T, H, dtype=torch.uint8, device="cuda")
    s = torch.empty(T, H // 128, device="cuda")
    inv = torch.empty(T, device="cuda")
    api.moe_rms_norm(x, None, w.cuda(), EPS, None, y, c, s, inv)
    v, dv, r, dr = plain.norm(x[at].double().cpu(), w.double(), EPS)
    check(y[at], v, plain.rounded16(v, dv), "y")
    check_codes(c[at], s[at], v, dv)
    gx, gw = torch.empty_like(x), torch.empty(H, device="cuda")
    api.moe_rms_norm_backward(x, x, w.cuda(), inv, None, gx, gw)
    t = x[at].double().cpu()
    want_x, want_w = plain.norm_grad(t, t, w.double(), inv[at].double().cpu(), None)
    check(gx[at], *want_x, "grad_x")
    check(gw, want_w[0], want_w[1], "grad_weight")   # the other rows are zeros


# Thread layouts: a row to 16, 32, 64, 256 and 1024 threads, to kept and to reloaded rows.
LAYOUTS = [(1, 128), (60, 128), (60, 256), (60, 512), (60, 1024), (60, 2048), (300, 4096),
           (300, 8192), (60, 8320), (3, 16384), (60, 16512), (20, 32896), (20, 65536)]


@pytest.mark.parametrize("T,H", LAYOUTS)
@pytest.mark.parametrize("eps", [EPS, 0.0])
def test_norm_of_rows_whose_squares_leave_fp32(T, H, eps):
    """Rows of any finite values that bf16 holds: squares from 2^-240 to 2^252, one value
    among small ones, and the same through the gradient."""
    powers = [124, 120, 70, 64, 63, 60, 56, 20, -60, -70, -110, -120]
    gen = torch.Generator().manual_seed(T + H)
    x = torch.randn(T, H, generator=gen, dtype=torch.float64)
    x *= torch.tensor([2.0 ** powers[i % len(powers)] for i in range(T)]).double()[:, None]
    if T > 20:
        x[13], x[14] = x[13].sign(), x[14].sign()
        x[13, H // 2], x[14, 3] = 2.0 ** 100, -2.0 ** 118
        x[15], x[16] = -2.0 ** 127, 2.0 ** 64 / H ** 0.5
    x, w = x.bfloat16(), norm_weight(H, T)
    assert x.isfinite().all()
    y, c, s = out(T, H), out(T, H, torch.uint8), out(T, H // 128, torch.float32)
    inv = torch.full((T + 1,), FILL, device="cuda")
    api.moe_rms_norm(x.cuda(), None, w.cuda(), eps, None, y, c, s, inv)
    v, dv, r, dr = plain.norm(x.double(), w.double(), eps)
    check(inv[:T], r, dr, "1 / rms")
    check(y[:T], v, plain.rounded16(v, dv), "y")
    check_codes(c[:T], s[:T], v, dv)
    gy = (0.01 * torch.randn(T, H, generator=gen)).bfloat16()
    gx, gw = out(T, H), torch.empty(H, device="cuda")
    api.moe_rms_norm_backward(gy.cuda(), x.cuda(), w.cuda(), inv[:T], None, gx, gw)
    want_x, want_w = plain.norm_grad(gy.double(), x.double(), w.double(), inv[:T].double().cpu(), None)
    check(gx[:T], *want_x, "grad_x")
    check(gw, *want_w, "grad_weight")


def wide_rows(T, H, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, H, generator=gen, device="cuda").bfloat16()


def check_here(got, want, bound, what):
    off = (got.double() - want).abs()
    assert (off <= bound).all(), (what, float((off - bound).max()))


# Launches end at 1024 blocks forward and 512 back: past twice as many rows a group of 1024
# threads takes a third one, which uses the first one's places in LDS again.
@pytest.mark.parametrize("T,H", [(2100, 8200), (2051, 16384), (2100, 16392), (2060, 32776),
                                 (2049, 65536)])
def test_norm_of_several_wide_rows_a_block(T, H):
    x, res, w = wide_rows(T, H, 1), wide_rows(T, H, 2), norm_weight(H, T).cuda()
    total, y = torch.empty_like(x), torch.empty_like(x)
    inv = torch.empty(T, device="cuda")
    codes = H % 128 == 0
    c = torch.empty(T, H, dtype=torch.uint8, device="cuda") if codes else None
    s = torch.empty(T, H // 128, device="cuda") if codes else None
    api.moe_rms_norm(x, res, w, EPS, total, y, c, s, inv)
    assert torch.equal(total, (x.float() + res.float()).bfloat16())
    v, dv, r, dr = plain.norm(total.double(), w.double(), EPS)
    check_here(y, v, plain.rounded16(v, dv), "y")
    check_here(inv, r, dr, "1 / rms")
    if codes:
        at = [0, 1, 1023, 1024, 1025, 2047, 2048, T - 1]
        check_codes(c[at], s[at], v[at].cpu(), dv[at].cpu())
    # the residual stream in place, and the rows over the input's
    api.moe_rms_norm(x, res, w, EPS, res, x)
    assert torch.equal(res, total) and torch.equal(x, y)


@pytest.mark.parametrize("T,H", [(1100, 8200), (1030, 16384), (1100, 16392), (1030, 32776),
                                 (1025, 65536)])
def test_norm_gradient_of_several_wide_rows_a_block(T, H):
    t, gy, carried = wide_rows(T, H, 3), wide_rows(T, H, 4), wide_rows(T, H, 5)
    w = norm_weight(H, T).cuda()
    r = (t.double().square().mean(1) + EPS).rsqrt().float()
    gx, gw = torch.empty_like(t), torch.empty(H, device="cuda")
    api.moe_rms_norm_backward(gy, t, w, r, carried, gx, gw)
    want_x, want_w = plain.norm_grad(gy.double(), t.double(), w.double(), r.double(), carried.double())
    check_here(gx, *want_x, "grad_x")
    check_here(gw, *want_w, "grad_weight")
    again = torch.empty_like(gw)
    api.moe_rms_norm_backward(gy, t, w, r, carried, carried, again)
    assert torch.equal(carried, gx) and torch.equal(again, gw)
    api.moe_rms_norm_backward(gy, t, w, r, None, gx, None)
    api.moe_rms_norm_backward(gy, t, w, r, None, gy, again)
    assert torch.equal(gy, gx) and torch.equal(again, gw)


@pytest.mark.parametrize("T,H", [(3000, 512), (1100, 8192), (1030, 16384), (3, 40960)])
def test_norm_in_place_the_other_way(T, H):
    """total over the input and y over the residual."""
    x, res, w = wide_rows(T, H, 7), wide_rows(T, H, 8), norm_weight(H, 7).cuda()
    t, y = torch.empty_like(x), torch.empty_like(x)
    api.moe_rms_norm(x, res, w, EPS, t, y)
    api.moe_rms_norm(x, res, w, EPS, x, res)
    assert torch.equal(x, t) and torch.equal(res, y)
