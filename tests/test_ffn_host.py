"""Host-side refusals of include/moe_ffn.h (no GPU needed): every call returns the
documented status before any launch; the header's symbols are exported; the binding
refuses tensors that the kernels could run past.  And the plain gradients against
differences."""
import ctypes
import os
import re

import pytest
import torch

import ffn_reference as plain

api = pytest.importorskip("combine_moe_dispatch_amd.api",
                          reason="libmoe_dispatch.so not built")

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "moe_ffn.h")
A = 4096       # an aligned stand-in address, never touched on these paths
ODD = 4096 + 8
OK, INVALID, UNSUPPORTED = 0, 1, 2

GOOD = (4, 128, 8, 2, 2, 0, 1)
FFN = (128, 256)


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", text))
    assert {"moe_rms_norm", "moe_rms_norm_backward", "moe_quantize_weight", "moe_expert_ffn",
            "moe_expert_ffn_backward"} <= names
    for n in names:
        assert hasattr(api._lib, n), n


def norm(x=A, res=None, w=A, T=4, H=256, total=A, y=2 * A, codes=A, scales=A, inv=A):
    return api._lib.moe_rms_norm(x, res, w, T, H, 1e-6, total, y, codes, scales, inv, None)


def norm_grad(gy=A, t=A, w=A, inv=A, carried=None, T=4, H=256, gx=A, gw=A, ws=A, n=1 << 40):
    return api._lib.moe_rms_norm_backward(gy, t, w, inv, carried, T, H, gx, gw, ws, n, None)


@pytest.mark.parametrize("call", [norm, norm_grad])
def test_norm_sizes(call):
    assert call(T=-1) == INVALID
    for H in (0, -8, 12):
        assert call(H=H) == INVALID
    assert call(H=65536 + 128) == UNSUPPORTED
    for kw in (dict(w=None), dict(w=ODD)):
        assert call(**kw) == INVALID, kw


def test_norm_refusals():
    assert norm(total=None, y=None, codes=None, scales=None, inv=None) == INVALID
    assert norm(codes=None) == INVALID
    assert norm(scales=None) == INVALID
    assert norm(H=136) == INVALID                        # 8-bit rows in blocks of 128
    assert norm(total=A, y=A) == INVALID
    for kw in (dict(x=None), dict(x=ODD), dict(res=ODD), dict(total=ODD), dict(y=ODD),
               dict(codes=ODD)):
        assert norm(**kw) == INVALID, kw
    assert norm(T=0, x=None) == OK


def test_norm_grad_refusals():
    assert norm_grad(gx=None, gw=None) == INVALID
    for kw in (dict(gy=None), dict(gy=ODD), dict(t=None), dict(t=ODD), dict(inv=None),
               dict(carried=ODD), dict(gx=ODD), dict(gw=ODD), dict(ws=None), dict(ws=ODD)):
        assert norm_grad(**kw) == INVALID, kw
    need = api.moe_rms_norm_backward_workspace_size(4, 256)
    assert need > 0
    assert norm_grad(n=need - 1) == INVALID
    assert api.moe_rms_norm_backward_workspace_size(1, 256) == 0
    assert api.moe_rms_norm_backward_workspace_size(4, 12) == 0
    assert norm_grad(T=0, gw=None, gy=None) == OK


def weight(w=A, kind=0, E=2, P=128, K=256, codes=A, scales=A):
    return api._lib.moe_quantize_weight(w, kind, E, P, K, codes, scales, None)


def test_weight_refusals():
    for kw in (dict(kind=2), dict(kind=-1), dict(E=0), dict(P=0), dict(K=0), dict(P=64),
               dict(K=200), dict(w=None), dict(w=ODD), dict(codes=None), dict(codes=ODD),
               dict(scales=None)):
        assert weight(**kw) == INVALID, kw
    assert weight(E=1025) == UNSUPPORTED
    assert weight(K=(1 << 22) + 128) == UNSUPPORTED
    assert weight(E=1024, P=128 * 128, K=128 * 128) == UNSUPPORTED


def ref(c):
    return None if c is None else ctypes.byref(c)


def layout(counts=A, offsets=A):
    return api._Layout(counts, offsets, None, None, None, None, None)


def ffn(shape=GOOD, f=FFN, x=A, xs=A, lay=layout(), up=A, us=A, down=A, ds=A, res=None, y=A,
        pre=None, ws=A, n=1 << 60):
    return api._lib.moe_expert_ffn(
        ref(None if shape is None else api._Shape(*shape)),
        ref(None if f is None else api._Ffn(*f)), x, xs, ref(lay), up, us, down, ds, res, y, pre,
        ws, n, None)


def ffn_grad(shape=GOOD, f=FFN, gy=A, x=A, xs=A, lay=layout(), up=A, us=A, down=A, ds=A, pre=A,
             gx=A, gu=A, gd=A, ws=A, n=1 << 60):
    return api._lib.moe_expert_ffn_backward(
        ref(None if shape is None else api._Shape(*shape)),
        ref(None if f is None else api._Ffn(*f)), gy, x, xs, ref(lay), up, us, down, ds, pre, gx,
        gu, gd, ws, n, None)


@pytest.mark.parametrize("call", [ffn, ffn_grad])
def test_ffn_shapes(call):
    for shape, code in (((4, 128, 8, 9, 2, 0, 1), INVALID), ((4, 128, 9, 2, 2, 0, 1), INVALID),
                        ((-1, 128, 8, 2, 2, 0, 1), INVALID), ((4, 64, 8, 2, 2, 0, 1), INVALID),
                        ((4, 128, 8, 2, 2, 0, 3), INVALID), (None, INVALID),
                        ((4, 128, 8, 2, 2, 0, 0), UNSUPPORTED),          # bf16
                        ((4, 128, 2048, 2, 2, 0, 1), UNSUPPORTED),
                        ((1 << 30, 128, 8, 4, 2, 0, 1), UNSUPPORTED)):
        assert call(shape=shape) == code, shape
    for f in ((0, 128), (128, 0), (-128, 128), (64, 128), (128, 192), None):
        assert call(f=f) == INVALID, f
    assert call(f=((1 << 22) + 128, 128)) == UNSUPPORTED
    assert call(f=(128, (1 << 21) + 128)) == UNSUPPORTED
    assert call(lay=None) == INVALID                                      # several experts
    assert call(shape=(9, 128, 1, 1, 1, 4, 1), lay=None) == INVALID       # more tokens than rows
    assert call(lay=layout(counts=None)) == INVALID
    assert call(lay=layout(offsets=None)) == INVALID
    # more tiles than a launch has
    assert call(shape=(1 << 30, 128, 1, 1, 1, 0, 1), lay=None, f=(1 << 22, 128)) == UNSUPPORTED


def test_ffn_refusals():
    for kw in (dict(x=None), dict(x=ODD), dict(xs=None), dict(up=None), dict(up=ODD),
               dict(us=None), dict(down=None), dict(down=ODD), dict(ds=None), dict(res=ODD),
               dict(y=None), dict(y=ODD), dict(pre=ODD), dict(ws=None), dict(ws=ODD)):
        assert ffn(**kw) == INVALID, kw
    need = api.moe_expert_ffn_workspace_size(api.Shape(*GOOD), api.Ffn(*FFN))
    assert need >= 8 * 256
    assert ffn(n=need - 1) == INVALID
    assert ffn(shape=(0, 128, 8, 2, 2, 0, 1), x=None, y=None, ws=None) == OK
    assert api.moe_expert_ffn_workspace_size(api.Shape(4, 128, 8, 2, 2, 0, 0), api.Ffn(*FFN)) == 0


def test_ffn_grad_refusals():
    assert ffn_grad(gx=None, gu=None, gd=None) == INVALID
    for kw in (dict(gy=None), dict(gy=ODD), dict(x=None), dict(x=ODD), dict(xs=None),
               dict(up=None), dict(up=ODD), dict(us=None), dict(down=None), dict(down=ODD),
               dict(ds=None), dict(pre=None), dict(pre=ODD), dict(gx=ODD), dict(gu=ODD),
               dict(gd=ODD), dict(ws=None), dict(ws=ODD)):
        assert ffn_grad(**kw) == INVALID, kw
    need = api.moe_expert_ffn_backward_workspace_size(api.Shape(*GOOD), api.Ffn(*FFN))
    assert need >= 8 * (128 + 512 + 1024 + 512 + 256)
    assert ffn_grad(n=need - 1) == INVALID
    assert ffn_grad(shape=(0, 128, 8, 2, 2, 0, 1), gu=None, gd=None, ws=None) == OK
    # more tiles of the weights' gradients than can be numbered
    assert ffn_grad(shape=(4, 128, 1024, 2, 2, 0, 1), f=(1 << 22, 128 * 1024)) == UNSUPPORTED


def test_sums_in_shares_take_room_for_placed_rows_alone():
    """128 tokens of 8 experts each have 1024 rows, wherever in 32 regions of 4096 they lie."""
    H, I = 7168, 2048
    ffn = api.Ffn(H, I)
    packed = api.moe_expert_ffn_workspace_size(api.Shape(128, H, 256, 8, 32, 0, 1), ffn)
    fixed = api.moe_expert_ffn_workspace_size(api.Shape(128, H, 256, 8, 32, 4096, 1), ffn)
    row = I + I // 128 * 4    # the codes and scales between the projections
    assert packed >= 1024 * (row + 2 * I * 4)
    assert fixed - packed == (32 * 4096 - 1024) * row


def test_binding_refuses_before_any_launch():
    cpu = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256)
    with pytest.raises(ValueError, match="GPU tensor"):
        api.moe_rms_norm(cpu, None, w, 1e-6, None, cpu)
    with pytest.raises(ValueError, match="2-D"):
        api.moe_rms_norm(cpu[0], None, w, 1e-6, None, cpu)
    with pytest.raises(ValueError, match="GPU tensor"):
        api.moe_rms_norm_backward(cpu, cpu, w, w, None, cpu, None)
    with pytest.raises(ValueError, match=r"\[E, P, K\]"):
        api.moe_quantize_weight(w, w, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        api.moe_quantize_weight(cpu, cpu, w)
    shape, f = api.Shape(*GOOD), api.Ffn(*FFN)
    with pytest.raises(ValueError, match="x is required"):
        api.moe_expert_ffn(shape, f, None, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="grad_y is required"):
        api.moe_expert_ffn_backward(shape, f, None, None, None, None, None, None, None, None,
                                    None, None, None, None)
    with pytest.raises(api.MoeError):  # the library names a bad shape
        api.moe_expert_ffn(api.Shape(4, 128, 9, 2, 2, 0, 1), f, None, None, None, None, None,
                           None, None, None, None)


def test_plain_block_gradient_against_differences():
    """The formula of the gradients (roundings left out) against central differences."""
    torch.manual_seed(0)
    x, up, down = torch.randn(3, 8).double(), torch.randn(12, 8).double(), torch.randn(8, 6).double()
    gy = torch.randn(3, 8).double()
    silu = lambda v: v * torch.sigmoid(v)  # noqa: E731

    def loss(x, up, down):
        g, u = (x @ up.T).chunk(2, 1)
        return ((silu(g) * u) @ down.T * gy).sum()

    g, u = (x @ up.T).chunk(2, 1)
    s = torch.sigmoid(g)
    gh = gy @ down
    gz = torch.cat([gh * u * s * (1 + g * (1 - s)), gh * g * s], 1)
    grads = gz @ up, gz.T @ x, gy.T @ (g * s * u)
    for i, grad in enumerate(grads):
        args = [x, up, down]
        for at in ((0, 0), (2, 5), (1, 3)):
            d = torch.zeros_like(args[i])
            d[at] = 1e-5
            hi, lo = ([a + e * d if j == i else a for j, a in enumerate(args)] for e in (1, -1))
            assert abs((loss(*hi) - loss(*lo)) / 2e-5 - grad[at]) < 1e-7


def test_plain_norm_gradient_against_differences():
    torch.manual_seed(1)
    t, w, gy = torch.randn(3, 8).double(), torch.randn(8).double(), torch.randn(3, 8).double()
    loss = lambda t, w: (plain.norm(t, w, 1e-3)[0] * gy).sum()  # noqa: E731
    r = plain.norm(t, w, 1e-3)[2]
    (gx, _), (gw, _) = plain.norm_grad(gy, t, w, r, None)
    for at in ((0, 0), (2, 5), (1, 3)):
        d = torch.zeros_like(t)
        d[at] = 1e-5
        assert abs((loss(t + d, w) - loss(t - d, w)) / 2e-5 - gx[at]) < 1e-7
        e = torch.zeros_like(w)
        e[at[1]] = 1e-5
        assert abs((loss(t, w + e) - loss(t, w - e)) / 2e-5 - gw[at[1]]) < 1e-7


def test_plain_codes():
    """The rounding to e4m3 against torch's cast, every code and every border."""
    all_codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    v = all_codes[all_codes.isfinite()].sort().values
    border = (v[1:] + v[:-1]) / 2
    for q in (v, border, border * (1 + 2.0 ** -20), border * (1 - 2.0 ** -20)):
        assert torch.equal(plain.e4m3(q), q.float().to(torch.float8_e4m3fn).double())
    r = torch.randn(7, 256)
    codes, scales = plain.codes_of(r)
    assert (codes.abs().amax(1) == 448).all()
    value, slack = plain.quantize(r.double(), torch.zeros(7, 256, dtype=torch.float64))
    again = (codes.unflatten(-1, (-1, 128)) * scales.double()[..., None]).flatten(-2)
    assert ((value - again).abs() <= slack + 1e-30).all()
