"""The expert product and its gradients past 2^31 entries of experts times
columns (35 GB of weights)."""
import pytest
import torch

import expert_reference as ref
from combine_moe_dispatch_amd import api

pytestmark = pytest.mark.gpu

FILL = -7.0


def test_more_columns_of_all_experts_than_31_bits():
    E, P, K = 520, 1 << 22, 8
    assert E * P > 1 << 31
    shape = api.Shape(1, K, E, 2, 1, 0)
    lin = api.Linear(K, P)
    gen = torch.Generator().manual_seed(5)
    busy = (3, 519)
    counts = torch.zeros(E, dtype=torch.int32)
    counts[list(busy)] = 1
    offsets = (counts.cumsum(0) - counts).int().cuda()
    lay = api.Layout(counts.cuda(), offsets, None, None, None, None, None)
    w = torch.zeros(E, P, K, dtype=torch.bfloat16, device="cuda")
    own = torch.randn(2, P, K, generator=gen).bfloat16()
    w[list(busy)] = own.cuda()
    x = torch.randn(2, K, generator=gen).bfloat16()
    y = torch.full((3, P), FILL, dtype=torch.bfloat16, device="cuda")
    api.moe_expert_matmul(shape, lin, x.cuda(), None, lay, w, None, None, None, y)
    spans = [(0, 1), (1, 2)]
    want = ref.matmul(x.double(), own.double(), None, None, spans, "none", P)
    ref.check(y[:2], want[0], want[2], "y")
    assert (y[2] == FILL).all()

    gy = torch.randn(2, P, generator=gen).bfloat16()
    gx = torch.full((3, K), FILL, dtype=torch.bfloat16, device="cuda")
    gw = torch.full_like(w, FILL)
    api.moe_expert_matmul_backward(shape, lin, gy.cuda(), x.cuda(), lay, w, None, gx, gw, None)
    (wx, ww, _), (tx, tw, _) = ref.matmul_grad(gy.double(), x.double(), own.double(), None, spans,
                                               "none")
    ref.check(gx[:2], wx, tx, "grad_x")
    assert (gx[2] == FILL).all()
    for i, e in enumerate(busy):
        ref.check(gw[e], ww[i], tw[i], "grad_weight")
        gw[e].zero_()
    for e in range(0, E, 8):
        assert not gw[e:e + 8].any()
