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


@pytest.mark.parametrize("mean", [96, 102, 103, 128])
@pytest.mark.parametrize("name", ["none", "swiglu"])
def test_fp8_rows_around_the_mean(mean, name):
    """Experts with more and fewer rows than the mean, on both sides of the rule that
    takes 128 x 128 tiles: to the bit what each expert's rows give alone."""
    E, K = 8, 256
    F = 2304 // (2 if name == "swiglu" else 1)
    P = 2304
    counts = mean + torch.tensor([0, 12, -12, 33, -33, 1, -1, 0])
    R = int(counts.sum())
    gen = torch.Generator(device="cuda").manual_seed(mean)
    u8 = lambda *s: torch.randint(0, 120, s, dtype=torch.uint8, device="cuda", generator=gen)  # noqa: E731
    f32 = lambda *s: torch.rand(*s, device="cuda", generator=gen) / 64  # noqa: E731
    x, xs, w, ws = u8(R, K), f32(R, K // 128), u8(E, P, K), f32(E, P // 128, K // 128)
    offsets = counts.cumsum(0) - counts
    lay = api.Layout(counts.int().cuda(), offsets.int().cuda(), None, None, None, None, None)
    lin = api.Linear(K, F, {"none": api.MOE_ACT_NONE, "swiglu": api.MOE_ACT_SWIGLU}[name])
    y = torch.full((R + 2, F), FILL, dtype=torch.bfloat16, device="cuda")
    api.moe_expert_matmul(api.Shape(R, K, E, 1, 1, 0, 1), lin, x, xs, lay, w, ws, None, None, y)
    assert (y[R:] == FILL).all()
    for e, (a, n) in enumerate(zip(offsets.tolist(), counts.tolist())):
        alone = torch.empty(n, F, dtype=torch.bfloat16, device="cuda")
        api.moe_expert_matmul(api.Shape(n, K, 1, 1, 1, 0, 1), lin, x[a:a + n].contiguous(),
                              xs[a:a + n].contiguous(), None, w[e].contiguous(),
                              ws[e].contiguous(), None, None, alone)
        assert torch.equal(y[a:a + n], alone), e
