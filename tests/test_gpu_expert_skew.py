"""The expert product with rows bunched in a few of many experts, on both sides
of the rule that takes the streaming product (128 rows)."""
import pytest
import torch

import expert_reference as ref
from combine_moe_dispatch_amd import api

pytestmark = pytest.mark.gpu

FILL = -7.0


def bunched(E, R, kind):
    c = torch.zeros(E, dtype=torch.int64)
    if kind == "one":
        c[E - 1] = R
    elif kind == "eight":
        c[3:3 + 8] = R // 8
        c[3] += R % 8
    elif kind == "hot":
        c[7] = R // 2
        c[8:8 + R - R // 2] = 1
    return c


@pytest.mark.parametrize("kind", ["one", "eight", "hot"])
@pytest.mark.parametrize("E,R", [(64, 64), (64, 128), (64, 129), (70, 255), (300, 600)])
@pytest.mark.parametrize("K,F,name", [(72, 520, "none"), (136, 264, "swiglu")])
def test_bunched_rows(E, R, kind, K, F, name):
    R = min(R, 2 * (E - 8)) if kind == "hot" else R
    counts = bunched(E, R, kind)
    assert int(counts.sum()) == R
    P = F * (2 if name == "swiglu" else 1)
    gen = torch.Generator().manual_seed(E + R)
    x = torch.randn(R, K, generator=gen).bfloat16()
    w = (torch.randn(E, P, K, generator=gen) * K ** -0.5).bfloat16()
    b = torch.randn(E, P, generator=gen)
    offsets = counts.cumsum(0) - counts
    lay = api.Layout(counts.int().cuda(), offsets.int().cuda(), None, None, None, None, None)
    y = torch.full((R + 2, F), FILL, dtype=torch.bfloat16, device="cuda")
    act = {"none": api.MOE_ACT_NONE, "swiglu": api.MOE_ACT_SWIGLU}[name]
    api.moe_expert_matmul(api.Shape(R, K, E, 1, 1, 0), api.Linear(K, F, act), x.cuda(), None, lay,
                          w.cuda(), None, b.cuda(), None, y)
    spans = ref.segments(counts.tolist(), offsets.tolist(), E, 0)
    want = ref.matmul(x.double(), w.double(), b.double(), None, spans, name, F)
    ref.check(y[:R], want[0], want[2], "y", FILL)
    assert (y[R:] == FILL).all()
