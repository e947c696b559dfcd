"""Host-side refusals of include/moe_experts.h (no GPU needed): every call
returns the documented status before any launch; the header's symbols are
exported; the binding refuses tensors the kernels could run past."""
import ctypes
import os
import re

import pytest
import torch

api = pytest.importorskip("combine_moe_dispatch_amd.api",
                          reason="libmoe_dispatch.so not built")

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "moe_experts.h")
A = 4096       # an aligned stand-in address, never touched on these paths
ODD = 4096 + 8
INVALID, UNSUPPORTED = 1, 2

GOOD = (4, 64, 8, 2, 2, 0, 0)
LIN = (64, 32, 0)


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", text))
    assert {"moe_expert_matmul", "moe_expert_matmul_backward", "moe_combine_backward",
            "moe_balance_loss", "moe_route_backward"} <= names
    for n in names:
        assert hasattr(api._lib, n), n


def layout(counts=A, offsets=A, token_row=A):
    return api._Layout(counts, offsets, None, None, token_row, None, None)


def matmul(shape=GOOD, lin=LIN, x=A, xs=None, lay=layout(), w=A, ws=None, bias=None, res=None,
           y=A, pre=None):
    return api._lib.moe_expert_matmul(
        None if shape is None else ctypes.byref(api._Shape(*shape)),
        None if lin is None else ctypes.byref(api._Linear(*lin)), x, xs,
        None if lay is None else ctypes.byref(lay), w, ws, bias, res, y, pre, None)


BAD_SHAPES = [((4, 64, 8, 9, 2, 0, 0), INVALID), ((4, 64, 9, 2, 2, 0, 0), INVALID),
              ((-1, 64, 8, 2, 2, 0, 0), INVALID), ((4, 12, 8, 2, 2, 0, 0), INVALID),
              ((4, 64, 8, 2, 2, 0, 3), INVALID), ((4, 64, 2048, 2, 2, 0, 0), UNSUPPORTED),
              ((4, 64, 64, 33, 2, 0, 0), UNSUPPORTED),
              ((1 << 30, 64, 8, 4, 2, 0, 0), UNSUPPORTED)]
BAD_LINEARS = [(0, 32, 0), (64, 0, 0), (-8, 32, 0), (60, 32, 0), (64, 36, 0), (64, 32, 4),
               (64, 32, -1)]


@pytest.mark.parametrize("shape,code", BAD_SHAPES)
def test_bad_shapes(shape, code):
    assert matmul(shape=shape) == code
    assert backward(shape=shape) == code
    assert combine(shape=shape) == code
    s = ctypes.byref(api._Shape(*shape))
    assert api._lib.moe_expert_matmul_backward_workspace_size(
        s, ctypes.byref(api._Linear(*LIN))) == 0


@pytest.mark.parametrize("lin", BAD_LINEARS)
def test_bad_linears(lin):
    assert matmul(lin=lin) == INVALID
    assert backward(lin=lin) == INVALID


def test_matmul_refusals():
    assert matmul(shape=None) == INVALID
    assert matmul(lin=None) == INVALID
    assert matmul(lay=None) == INVALID                      # several experts need a layout
    assert matmul(shape=(9, 64, 1, 1, 1, 4, 0), lay=None) == INVALID  # more tokens than rows
    assert matmul(lay=layout(counts=None)) == INVALID
    assert matmul(lay=layout(offsets=None)) == INVALID
    for kw in (dict(x=None), dict(x=ODD), dict(w=None), dict(w=ODD), dict(y=None), dict(y=ODD),
               dict(bias=ODD), dict(res=ODD), dict(pre=ODD)):
        assert matmul(**kw) == INVALID, kw
    fp8 = (4, 128, 8, 2, 2, 0, 1)
    assert matmul(shape=fp8, lin=(128, 128, 0), xs=None, ws=A) == INVALID
    assert matmul(shape=fp8, lin=(128, 128, 0), xs=A, ws=None) == INVALID
    assert matmul(shape=fp8, lin=(64, 128, 0), xs=A, ws=A) == INVALID
    assert matmul(shape=fp8, lin=(128, 64, 0), xs=A, ws=A) == INVALID
    assert matmul(lin=(64, 1 << 30, 3)) == UNSUPPORTED
    assert matmul(lin=((1 << 22) + 8, 32, 0)) == UNSUPPORTED
    assert matmul(lin=(64, (1 << 21) + 8, 3)) == UNSUPPORTED
    assert matmul(shape=(0, 64, 8, 2, 2, 0, 0), x=None, w=None, y=None) == 0  # nothing to do


def backward(shape=GOOD, lin=LIN, gy=A, x=A, lay=layout(), w=A, pre=A, gx=A, gw=A, gb=A, ws=A,
             n=1 << 40):
    return api._lib.moe_expert_matmul_backward(
        None if shape is None else ctypes.byref(api._Shape(*shape)),
        None if lin is None else ctypes.byref(api._Linear(*lin)), gy, x,
        None if lay is None else ctypes.byref(lay), w, pre, gx, gw, gb, ws, n, None)


def test_backward_refusals():
    silu = (64, 32, 1)
    assert backward(shape=(4, 128, 8, 2, 2, 0, 1), lin=(128, 128, 0)) == UNSUPPORTED  # fp8
    assert backward(gx=None, gw=None, gb=None) == INVALID
    for kw in (dict(gy=None), dict(gy=ODD), dict(x=None), dict(x=ODD), dict(w=None), dict(w=ODD),
               dict(gx=ODD), dict(gw=ODD), dict(gb=ODD), dict(lay=None)):
        assert backward(**kw) == INVALID, kw
    assert backward(lin=silu, pre=None) == INVALID
    assert backward(lin=silu, pre=ODD) == INVALID
    assert backward(lin=silu, ws=None) == INVALID
    assert backward(lin=silu, ws=ODD) == INVALID
    need = api.moe_expert_matmul_backward_workspace_size(api.Shape(*GOOD), api.Linear(*silu))
    assert need >= 8 * 32 * 2
    assert backward(lin=silu, n=need - 1) == INVALID


def combine(shape=GOOD, go=A, y=A, lay=layout(), w=A, gy=A, gw=A):
    return api._lib.moe_combine_backward(ctypes.byref(api._Shape(*shape)), go, y,
                                         None if lay is None else ctypes.byref(lay), w, gy, gw,
                                         None)


def test_combine_refusals():
    assert combine(shape=(4, 128, 8, 2, 2, 0, 1)) == UNSUPPORTED
    assert combine(gy=None, gw=None) == INVALID
    for kw in (dict(go=None), dict(go=ODD), dict(y=None), dict(y=ODD), dict(lay=None),
               dict(lay=layout(token_row=None)), dict(w=None), dict(gy=ODD)):
        assert combine(**kw) == INVALID, kw
    assert combine(shape=(0, 64, 8, 2, 2, 0, 0), go=None, y=None, lay=None) == 0


def balance(l=A, b=None, ids=A, T=4, E=8, k=2, score=1, off=None, S=1, c=A, p=A, n=A, loss=A,
            ws=A, size=1 << 40):
    return api._lib.moe_balance_loss(l, b, ids, T, E, k, score, off, S, 0.1, c, p, n, loss, ws,
                                     size, None)


def route(l=A, b=None, ids=A, w=A, gw=A, T=4, E=8, k=2, score=1, off=None, S=1, c=A, n=A, gl=None,
          out=A, gb=A, ws=A, size=1 << 40):
    return api._lib.moe_route_backward(l, b, ids, w, gw, T, E, k, score, off, S, 0.1, c, n, gl,
                                       out, gb, ws, size, None)


@pytest.mark.parametrize("call", [balance, route])
def test_router_refusals(call):
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(score=2), dict(S=0),
               dict(l=None), dict(ids=None), dict(S=2)):
        assert call(**kw) == INVALID, kw
    assert call(E=1025) == UNSUPPORTED
    assert call(E=64, k=33) == UNSUPPORTED
    assert call(E=1024, S=1 << 21, off=A) == UNSUPPORTED
    assert call(T=1 << 30, k=4) == UNSUPPORTED


def test_balance_and_route_pointers():
    for kw in (dict(c=None), dict(p=None), dict(n=None), dict(loss=None)):
        assert balance(**kw) == INVALID, kw
    for kw in (dict(c=None), dict(n=None), dict(c=None, n=None, gw=None), dict(w=None),
               dict(out=None)):
        assert route(**kw) == INVALID, kw
    need = api.moe_balance_loss_workspace_size(20000, 256, 3)
    if need:
        big = dict(T=20000, E=256, S=3, off=A)
        assert balance(**big, ws=None) == INVALID
        assert balance(**big, ws=ODD) == INVALID
        assert balance(**big, size=need - 1) == INVALID
    need = api.moe_route_backward_workspace_size(20000, 256)
    if need:
        assert route(T=20000, E=256, ws=None) == INVALID
        assert route(T=20000, E=256, ws=ODD) == INVALID
        assert route(T=20000, E=256, size=need - 1) == INVALID
    assert api.moe_balance_loss_workspace_size(-1, 8, 1) == 0
    assert api.moe_route_backward_workspace_size(4, 0) == 0


def test_binding_refuses_cpu_tensors():
    s = api.Shape(4, 64, 2, 1, 1, 0)
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    lay = api.Layout(*(torch.zeros(8, dtype=torch.int32) for _ in range(5)), None,
                     torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU tensor"):
        api.moe_expert_matmul(s, api.Linear(64, 64), t, None, lay, t, None, None, None, t)
    with pytest.raises(ValueError, match="is required"):
        api.moe_expert_matmul(s, api.Linear(64, 64), None, None, lay, None, None, None, None, None)
    with pytest.raises(ValueError, match="GPU tensor"):
        api.moe_combine_backward(s, t, t, lay, None, None, torch.zeros(4, 1))
    with pytest.raises(ValueError, match="layout is required"):
        api.moe_combine_backward(s, t, t, None, None, None, None)
    with pytest.raises(ValueError, match="GPU tensor"):
        api.moe_balance_loss(torch.zeros(4, 8), None, torch.zeros(4, 2, dtype=torch.int32), 1, 0.1)
    with pytest.raises(ValueError, match="2-D"):
        api.moe_route_backward(torch.zeros(8), None, torch.zeros(4, 2), None, None, 1)
    with pytest.raises(ValueError, match="2-D"):
        api.moe_balance_loss(torch.zeros(4, 8), None, torch.zeros(3, 2, dtype=torch.int32), 1, 0.1)
    with pytest.raises(ValueError, match="one sequence"):
        api.moe_balance_loss(torch.zeros(4, 8), None, torch.zeros(4, 2, dtype=torch.int32), 1, 0.1,
                             torch.zeros(1, dtype=torch.int32))
    with pytest.raises(api.MoeError):  # the library names what is wrong with the shape
        api.moe_expert_matmul(api.Shape(4, 64, 9, 2, 2, 0), api.Linear(64, 64), t, None, lay, t,
                              None, None, None, t)


def test_sizes_past_the_last_32_bit_row():
    """Rows and tokens whose tiles' numbers would pass 2^31, and grids a launch
    cannot have: refused before anything is launched."""
    most = (1 << 31) - 65536
    for rows in (most + 1, (1 << 31) - 1):
        shape = (rows, 8, 1, 1, 1, 0, 0)
        assert matmul(shape=shape) == UNSUPPORTED
        assert backward(shape=shape) == UNSUPPORTED
        assert combine(shape=shape) == UNSUPPORTED
    for call in (balance, route):
        assert call(T=(1 << 30) + 1, E=1, k=1) == UNSUPPORTED
    assert balance(E=1, k=1, S=(1 << 30) + 1, off=A) == UNSUPPORTED
    assert matmul(shape=(65536, 64, 1024, 32, 2, 0, 0), lin=(8, 1 << 22, 0)) == UNSUPPORTED
    assert backward(shape=(1, 64, 1024, 32, 2, 0, 0), lin=(8, 1 << 22, 0)) == UNSUPPORTED
