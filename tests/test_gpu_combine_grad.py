"""The combine's gradient against fp64: bit-exact rows, dot products within the
bound of an fp32 sum, skipped pairs, canaries."""
import pytest
import torch

from combine_moe_dispatch_amd import api, inputs
from expert_reference import U32

pytestmark = pytest.mark.gpu


def case(T, H, E, k, N, C, seed=0, bad=False):
    shape = api.Shape(T, H, E, k, N, C)
    ids = torch.from_numpy(inputs.random_ids(T, k, E, seed, distinct=k <= E)).cuda()
    if bad:
        ids[::3, 0] = E
        ids[1::4] = -1
    lay = api.Layout.empty(shape, "cuda")
    recv, _ = api.alloc_recv(shape, "cuda")
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=gen).bfloat16().cuda()
    api.moe_dispatch(shape, x, ids, recv, None, lay, api.alloc_workspace(shape, "cuda"))
    rows = recv.shape[0]
    y = torch.randn(rows, H, generator=gen).bfloat16().cuda()
    used = lay.token_row.flatten()
    free = torch.ones(rows + 1, dtype=torch.bool, device="cuda")
    free[used[used >= 0].long()] = False
    y[free[:rows]] = float("nan")  # rows of no pair must not matter
    go = torch.randn(T, H, generator=gen).bfloat16().cuda()
    w = torch.from_numpy(inputs.random_weights(T, k, seed)).cuda()
    return shape, lay, y, go, w


@pytest.mark.parametrize("T,H,E,k,N,C,bad", [
    (1, 8, 1, 1, 1, 0, False), (1, 7168, 256, 8, 32, 8, False), (16, 256, 8, 2, 2, 32, False),
    (100, 2048 + 8, 16, 3, 4, 40, True), (33, 520, 64, 32, 8, 0, False),
    (50, 32768, 8, 4, 1, 0, True), (1500, 64, 32, 7, 8, 0, True), (9, 136, 4, 4, 2, 1, False),
])
def test_gradients(T, H, E, k, N, C, bad):
    shape, lay, y, go, w = case(T, H, E, k, N, C, T + k, bad)
    rows = y.shape[0]
    gy = torch.full((rows + 2, H), -7.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.full((T + 1, k), -7.0, device="cuda")
    api.moe_combine_backward(shape, go, y, lay, w, gy, gw)
    row = lay.token_row.cpu().long()
    want = torch.full((rows + 2, H), -7.0, dtype=torch.bfloat16)
    t, j = (row >= 0).nonzero(as_tuple=True)
    g64, y64 = go.cpu().double(), y.cpu().double()
    # one fp32 product, then the nearest bf16
    want[row[t, j]] = (w.cpu()[t, j][:, None] * go.cpu()[t].float()).bfloat16()
    assert torch.equal(gy.cpu().view(torch.int16), want.view(torch.int16))
    prod = g64[t] * y64[row[t, j]]
    dots = torch.zeros(T, k, dtype=torch.float64)
    bound = torch.zeros(T, k, dtype=torch.float64)
    dots[t, j] = prod.sum(1)
    bound[t, j] = (H + 8) * U32 * prod.abs().sum(1)
    assert ((gw[:T].cpu().double() - dots).abs() <= bound).all()
    assert (gw[T:] == -7.0).all()
    # either output alone
    gy2, gw2 = torch.full_like(gy, -7.0), torch.full_like(gw, -7.0)
    api.moe_combine_backward(shape, go, None, lay, w, gy2, None)
    api.moe_combine_backward(shape, go, y, lay, None, None, gw2)
    assert torch.equal(gy2.view(torch.int16), gy.view(torch.int16)) and torch.equal(gw2, gw)


def test_no_tokens():
    shape = api.Shape(0, 64, 4, 2, 2, 8)
    lay = api.Layout.empty(shape, "cuda")
    gy = torch.full((16, 64), -7.0, dtype=torch.bfloat16, device="cuda")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    api.moe_combine_backward(shape, e, gy.clone(), lay, torch.empty(0, 2, device="cuda"), gy, None)
    assert (gy == -7.0).all()


def test_special_values():
    shape, lay, y, go, w = case(6, 72, 4, 2, 1, 0, 3)
    go[2, 71] = float("inf")
    go[4, 0] = float("nan")
    gy, gw = torch.zeros_like(y), torch.empty(6, 2, device="cuda")
    api.moe_combine_backward(shape, go, y, lay, w, gy, gw)
    assert gw[4].isnan().all() and gw[[0, 1, 3, 5]].isfinite().all()
    assert gw[2].isinf().all()
    rows = lay.token_row[[0, 1, 3, 5]].flatten().long()
    assert gy[rows].isfinite().all()


def test_more_pairs_than_one_launch_has_blocks():
    """2^24 pairs and some: every one once."""
    T, k = (1 << 21) + 3, 8
    shape = api.Shape(T, 8, 8, k, 1, 0)
    lay = api.Layout.empty(shape, "cuda")
    rows = T * k
    # token t's slot j in row (t, j) of the reversed order; every seventh pair skipped
    row = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda").view(T, k)
    skip = torch.arange(rows, device="cuda").view(T, k) % 7 == 3
    lay.token_row.copy_(torch.where(skip, -1, row))
    go = torch.randint(-8, 9, (T, 8), device="cuda").bfloat16()
    y = torch.randint(-8, 9, (rows, 8), device="cuda").bfloat16()
    w = torch.randint(1, 5, (T, k), device="cuda").float()
    gy = torch.full((rows, 8), -77.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.empty(T, k, device="cuda")
    api.moe_combine_backward(shape, go, y, lay, w, gy, gw)
    # small integers: every product and sum is exact
    pairs = go.float()[:, None, :].expand(T, k, 8)
    want = torch.where(skip[..., None], -77.0, pairs * w[..., None]).view(rows, 8).flip(0)
    assert torch.equal(gy.float(), want)
    dots = (pairs * y.float().flip(0).view(T, k, 8)).sum(2)
    assert torch.equal(gw, torch.where(skip, 0.0, dots))
