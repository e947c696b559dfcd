"""What the binding of moe_experts.h refuses on the GPU before any launch, and calls
whose first use is inside a capture."""
import subprocess
import sys

import pytest
import torch

from combine_moe_dispatch_amd import api

pytestmark = pytest.mark.gpu

DEV = "cuda"


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16, device=DEV)


def lay(E, T):
    z = torch.zeros(E, dtype=torch.int32, device=DEV)
    return api.Layout(z, z, z, z, torch.zeros(T, 1, dtype=torch.int32, device=DEV), None, z)


def matmul(x=None, w=None, y=None, bias=None, layout=None, xs=None, pre=None):
    s = api.Shape(4, 64, 2, 1, 1, 0)
    api.moe_expert_matmul(s, api.Linear(64, 32), bf(4, 64) if x is None else x, xs,
                          lay(2, 4) if layout is None else layout,
                          bf(2, 32, 64) if w is None else w, None, bias, None,
                          bf(4, 32) if y is None else y, pre)


@pytest.mark.parametrize("kw,error", [
    (dict(x=bf), "TypeError"),
    (dict(x=lambda: bf(64, 4).t()), "ValueError"),              # not contiguous
    (dict(x=lambda: bf(3, 64)), "ValueError"),                  # too small
    (dict(x=lambda: bf(4, 64).half()), "TypeError"),            # fp16 is not bf16
    (dict(x=lambda: bf(4, 64).float()), "TypeError"),
    (dict(w=lambda: bf(2, 31, 64)), "ValueError"),
    (dict(y=lambda: bf(4, 31)), "ValueError"),
    (dict(bias=lambda: bf(2, 32)), "TypeError"),                # biases are fp32
    (dict(bias=lambda: torch.zeros(63, device=DEV)), "ValueError"),
    (dict(pre=lambda: bf(4, 31)), "ValueError"),
    (dict(x=lambda: torch.zeros(4, 64, dtype=torch.bfloat16)), "ValueError"),
    (dict(layout=lambda: lay(1, 4)), "ValueError"),
])
def test_matmul(kw, error):
    args = {k: (v if v is bf else v()) for k, v in kw.items()}
    with pytest.raises((TypeError, ValueError)) as info:
        matmul(**args)
    assert info.type.__name__ == error


def test_misaligned_rows():
    x = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(4, 64)
    with pytest.raises(api.MoeError):
        matmul(x=x)


def test_router():
    l, ids = torch.zeros(5, 8, device=DEV), torch.zeros(5, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        api.moe_balance_loss(l.double(), None, ids, 1, 0.1)
    with pytest.raises(TypeError):
        api.moe_balance_loss(l, None, ids.long(), 1, 0.1)
    with pytest.raises(ValueError):
        api.moe_balance_loss(l, torch.zeros(7, device=DEV), ids, 1, 0.1)
    with pytest.raises(TypeError):
        api.moe_balance_loss(l, None, ids, 1, 0.1, torch.tensor([0, 5], device=DEV))
    with pytest.raises(ValueError):
        api.moe_route_backward(l, None, ids, None, torch.zeros(5, 2, device=DEV), 1)
    with pytest.raises(api.MoeError):  # neither part wanted
        api.moe_route_backward(l, None, ids, None, None, 1)
    with pytest.raises(api.MoeError):  # counts without tokens
        api.moe_route_backward(l, None, ids, None, None, 1,
                               expert_counts=torch.zeros(1, 8, dtype=torch.int32, device=DEV))


FIRST = """
import sys, torch
sys.path.insert(0, ".")
from combine_moe_dispatch_amd import api
T, K, F = {T}, 128, 2048
x = torch.randn(T, K, device="cuda").bfloat16()
w = torch.randn(1, F, K, device="cuda").bfloat16()
y, gx = torch.zeros(T, F, device="cuda").bfloat16(), torch.zeros_like(x)
gw, gb = torch.zeros_like(w), torch.zeros(1, F, device="cuda")
s, lin = api.Shape(T, K, 1, 1, 1, 0), api.Linear(K, F)
ws = api.alloc_expert_workspace(s, lin, "cuda")
torch.cuda.synchronize()
def step():
    api.moe_expert_matmul(s, lin, x, None, None, w, None, None, None, y)
    api.moe_expert_matmul_backward(s, lin, y, x, None, w, None, gx, gw, gb, ws)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
for _ in range(3):
    y.zero_(); gx.zero_(); gw.zero_(); gb.zero_()
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, gx, gw, gb)]
    step()
    torch.cuda.synchronize()
    for a, b in zip(got, (y, gx, gw, gb)):
        assert torch.equal(a, b) and a.abs().sum() > 0
print("captured ok")
"""


@pytest.mark.parametrize("T", [3, 300])
def test_first_call_inside_a_capture(T):
    """A process whose first calls of these kernels are captured ones."""
    r = subprocess.run([sys.executable, "-c", FIRST.format(T=T)], capture_output=True, text=True,
                       timeout=100)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stderr[-2000:]
