"""The weight gradient's blocks take tile after tile, of full, nearly empty and
empty experts; both tile sizes on both sides of the rule between them."""
import pytest
import torch

from combine_moe_dispatch_amd import api
from expert_reference import TINY, U16, U32

pytestmark = pytest.mark.gpu

MIXED = [300, 0, 1, 65, 0, 0, 257, 192, 0, 31, 130]


def check(counts, K, P, seed):
    E, R = len(counts), sum(counts)
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=gen).bfloat16().cuda()
    gy = torch.randn(R, P, generator=gen).bfloat16().cuda()
    c = torch.tensor(counts, dtype=torch.int32)
    lay = api.Layout(c.cuda(), (c.cumsum(0) - c).int().cuda(), None, None, None, None, None)
    gw = torch.full((E + 1, P, K), -7.0, dtype=torch.bfloat16, device="cuda")
    api.moe_expert_matmul_backward(api.Shape(R, K, E, 1, 1, 0), api.Linear(K, P), gy, x, lay, None,
                                   None, None, gw, None)
    at = 0
    for e, n in enumerate(counts):
        if n == 0:
            assert not gw[e].any(), e
            continue
        a, b = gy[at:at + n].double().t().contiguous(), x[at:at + n].double()
        want = a @ b
        bound = (n + 8) * U32 * (a.abs() @ b.abs())
        bound += U16 * (want.abs() + bound) + TINY
        assert ((gw[e].double() - want).abs() <= bound).all(), e
        at += n
    assert (gw[E] == -7.0).all()


# 32 tiles of 256 x 256 an expert: a block's next tile is the next expert's.
# Whole tiles (every store counted by the next tile's first wait) and ragged ones.
@pytest.mark.parametrize("K,P", [(1024, 2048), (1000, 2024)])
@pytest.mark.parametrize("first", [0, 1, 5])
def test_experts_one_after_the_other(K, P, first):
    counts = MIXED[first:] + MIXED[:first]
    check(3 * counts, K, P, K + first)


@pytest.mark.parametrize("K,P", [(128, 1024), (136, 1000)])
def test_small_tiles_one_after_the_other(K, P):
    check(10 * MIXED, K, P, K)


@pytest.mark.parametrize("counts,K,P", [
    ([64], 2048, 6136), ([65], 2048, 6136),           # 192 large tiles, rows on both sides
    ([65], 2048, 5888), ([65], 2048, 5896),           # 184 and 192 of them
    ([130, 0], 1536, 4096), ([128, 0], 1536, 4096),   # the mean counts idle experts
    ([1], 8, 8), ([129], 264, 136),
])
def test_both_sides_of_the_tile_rule(counts, K, P):
    check(counts, K, P, P + sum(counts))
