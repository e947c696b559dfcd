"""The experts' matrix product and its gradient against plain fp64 forms: head
layouts of dispatch (packed, fixed and overflowing capacity, bad ids, empty and
hot experts), both payloads, every activation, odd sizes, poisoned rows."""
import pytest
import torch

import expert_reference as ref
from combine_moe_dispatch_amd import api, inputs

pytestmark = pytest.mark.gpu

ACT = {"none": 0, "silu": 1, "gelu": 2, "swiglu": 3}
FILL = -7.0  # what outputs hold before a call


def layout(T, E, k, N, C, K, seed, hot=None, bad=False, fp8=False, counts=None):
    """Rows dispatched by the library into a poisoned receive buffer.  counts:
    rows of each expert (k == 1)."""
    shape = api.Shape(T, K, E, k, N, C, 1 if fp8 else 0)
    ids = inputs.random_ids(T, k, E, seed, distinct=k <= E, hot=hot)
    ids = torch.from_numpy(ids).cuda()
    if counts is not None:
        ids = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).int().cuda().view(T, 1)
    if bad:
        ids[::3, 0] = E
        ids[1::5] = -1
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=gen).bfloat16().cuda()
    lay = api.Layout.empty(shape, "cuda")
    recv, scales = api.alloc_recv(shape, "cuda", fill=0x7F if fp8 else 0xFFFF)  # NaN
    api.moe_dispatch(shape, x, ids, recv, scales, lay, api.alloc_workspace(shape, "cuda"))
    spans = ref.segments(lay.expert_counts.tolist(), lay.expert_offsets.tolist(), E // N, C)
    return shape, lay, recv, scales, spans


def host(t):
    """fp64 values of a bf16 tensor (or of int16 bits)."""
    return t.view(torch.bfloat16).double().cpu()


def weights(E, P, K, seed, fp8):
    gen = torch.Generator().manual_seed(seed + 1)
    w = torch.randn(E, P, K, generator=gen) * K ** -0.5
    if not fp8:
        return w.bfloat16().cuda(), None
    b = w.view(E, P // 128, 128, K // 128, 128)
    s = b.abs().amax(dim=(2, 4)) / 448.0
    codes = (b / s[:, :, None, :, None]).reshape(E, P, K).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).cuda(), s.contiguous().cuda()


def run(T, E, k, N, C, K, F, name, fp8=False, bias=True, residual=True, pre=True, seed=0, **kw):
    P = F * (2 if name == "swiglu" else 1)
    shape, lay, recv, xs, spans = layout(T, E, k, N, C, K, seed, fp8=fp8, **kw)
    rows = recv.shape[0]
    w, ws = weights(E, P, K, seed, fp8)
    gen = torch.Generator().manual_seed(seed + 2)
    b = torch.randn(E, P, generator=gen).cuda() if bias else None
    r = torch.randn(rows, F, generator=gen).bfloat16().cuda() if residual else None
    y = torch.full((rows + 3, F), FILL, dtype=torch.bfloat16, device="cuda")
    z = torch.full((rows + 3, P), FILL, dtype=torch.bfloat16, device="cuda") if pre else None
    api.moe_expert_matmul(shape, api.Linear(K, F, ACT[name]), recv, xs, lay, w, ws, b, r, y, z)
    x64 = ref.widen(recv.cpu(), xs.cpu(), 1) if fp8 else host(recv)
    w64 = ref.widen(w.cpu(), ws.cpu(), 128) if fp8 else host(w)
    want = ref.matmul(x64, w64, None if b is None else b.double().cpu(),
                      None if r is None else host(r), spans, name, F)
    ref.check(y[:rows], want[0], want[2], "y", FILL)
    assert (y[rows:] == FILL).all()
    if pre:
        ref.check(z[:rows], want[1], want[3], "pre", FILL)
        assert (z[rows:] == FILL).all()
    return y[:rows]


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("T,E,k,N,C,K,F", [
    (1, 8, 2, 2, 4, 64, 32),         # one token
    (16, 8, 2, 2, 32, 256, 64),      # fixed capacity, rows nobody reaches
    (37, 5, 3, 1, 0, 72, 40),        # packed, odd sizes
    (64, 4, 2, 2, 20, 8, 8),         # capacity overflows; the smallest row
    (130, 3, 1, 1, 0, 1432, 24),     # long reduction with a ragged end
])
def test_bf16(name, T, E, k, N, C, K, F):
    run(T, E, k, N, C, K, F, name)


@pytest.mark.parametrize("bias,residual,pre", [(False, False, False), (True, False, False),
                                               (False, True, True)])
@pytest.mark.parametrize("name", ["none", "swiglu"])
def test_optional_arguments(name, bias, residual, pre):
    run(33, 4, 2, 1, 0, 96, 48, name, bias=bias, residual=residual, pre=pre)


@pytest.mark.parametrize("name,T,E,k,N,C,K,F", [
    ("none", 1, 4, 1, 1, 0, 128, 128),
    ("silu", 50, 4, 2, 2, 30, 384, 256),
    ("gelu", 70, 2, 2, 1, 0, 128, 384),
    ("swiglu", 45, 3, 2, 1, 0, 640, 128),
    ("swiglu", 200, 2, 1, 2, 90, 256, 256),
    ("none", 600, 3, 2, 1, 0, 512, 640),
    ("swiglu", 600, 3, 2, 1, 0, 384, 384),
    ("swiglu", 2100, 1, 1, 1, 0, 128, 4096),  # enough rows and columns for the largest tiles
    ("none", 1100, 2, 1, 1, 0, 256, 8320),
    ("silu", 1500, 5, 2, 1, 0, 128, 3456),
])
def test_fp8(name, T, E, k, N, C, K, F):
    run(T, E, k, N, C, K, F, name, fp8=True)


@pytest.mark.parametrize("T", [15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_rows_around_the_tiles(T):
    run(T, 1, 1, 1, 0, 128, 264, "none", seed=T)
    run(T, 1, 1, 1, 0, 200, 136, "swiglu", seed=T)


@pytest.mark.parametrize("F", [8, 56, 64, 72, 120, 128, 136, 248, 256, 264])
def test_columns_around_the_tiles(F):
    run(90, 2, 1, 1, 0, 64, F, "silu", seed=F)
    run(300, 2, 2, 1, 0, 64, F, "swiglu", seed=F)


@pytest.mark.parametrize("K", [8, 16, 24, 32, 40, 56, 64, 72, 120, 128, 136, 192, 504, 512, 520])
def test_reductions_around_the_steps(K):
    run(20, 2, 1, 1, 0, K, 40, "none", seed=K)
    run(530, 2, 1, 1, 0, K, 72, "swiglu", seed=K)


@pytest.mark.parametrize("kw", [dict(hot=2), dict(bad=True), dict(hot=0, bad=True)])
def test_skew_and_bad_ids(kw):
    run(150, 8, 2, 4, 60, 64, 48, "swiglu", **kw)
    run(400, 8, 2, 1, 0, 64, 48, "none", **kw)


def test_no_tokens_writes_nothing():
    shape = api.Shape(0, 64, 4, 2, 2, 8)
    lay = api.Layout.empty(shape, "cuda")
    for f in ("expert_counts", "expert_offsets"):
        getattr(lay, f).zero_()
    z = lambda *s: torch.full(s, FILL, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y = z(16, 32)
    api.moe_expert_matmul(shape, api.Linear(64, 32), z(16, 64), None, lay, z(4, 32, 64), None,
                          None, None, y)
    assert (y == FILL).all()
    gw, gb = z(4, 32, 64), torch.full((4, 32), FILL, device="cuda")
    api.moe_expert_matmul_backward(shape, api.Linear(64, 32), z(16, 32), z(16, 64), lay,
                                   z(4, 32, 64), None, None, gw, gb)
    assert (gw == 0).all() and (gb == 0).all()


def test_all_ids_bad():
    """Every pair skipped: no row is read or written, gradients of weights are zero."""
    shape, lay, recv, _, spans = layout(20, 4, 2, 1, 0, 64, 3)
    lay.expert_counts.zero_()
    y = torch.full((40, 32), FILL, dtype=torch.bfloat16, device="cuda")
    w, _ = weights(4, 32, 64, 0, False)
    api.moe_expert_matmul(shape, api.Linear(64, 32), recv, None, lay, w, None, None, None, y)
    assert (y == FILL).all()
    gw = torch.full((4, 32, 64), FILL, dtype=torch.bfloat16, device="cuda")
    api.moe_expert_matmul_backward(shape, api.Linear(64, 32), y, recv, lay, None, None, None, gw,
                                   None)
    assert (gw == 0).all()


@pytest.mark.parametrize("T", [1, 3, 40, 300])
def test_dense_without_layout(T):
    """layout None: all rows belong to one expert; equal to the same call with a layout."""
    K, F = 136, 72
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, K, generator=gen).bfloat16().cuda()
    w, _ = weights(1, F, K, T, False)
    r = torch.randn(T, F, generator=gen).bfloat16().cuda()
    shape = api.Shape(T, K, 1, 1, 1, 0)
    y = r.clone()  # the residual may be the output itself
    api.moe_expert_matmul(shape, api.Linear(K, F, ACT["silu"]), x, None, None, w, None, None, y, y)
    want = ref.matmul(host(x), host(w), None, host(r), [(0, T)], "silu", F)
    ref.check(y, want[0], want[2], "y")
    lay = api.Layout.empty(shape, "cuda")
    lay.expert_counts.fill_(T)
    lay.expert_offsets.zero_()
    again = torch.empty_like(y)
    api.moe_expert_matmul(shape, api.Linear(K, F, ACT["silu"]), x, None, lay, w, None, None, r,
                          again)
    assert torch.equal(y, again)


def test_special_values():
    """NaN and infinities stay in the rows and columns that hold them."""
    T, K, F = 70, 64, 80
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = torch.randn(1, F, K, generator=gen).bfloat16()
    x[5, 63] = float("nan")
    x[69, 0] = float("inf")
    w[0, 79, 63] = float("inf")
    shape = api.Shape(T, K, 1, 1, 1, 0)
    y = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    api.moe_expert_matmul(shape, api.Linear(K, F), x.cuda(), None, None, w.cuda(), None, None,
                          None, y)
    want = x.double() @ w[0].double().T
    got = y.double().cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.isinf(), want.isinf())
    assert torch.equal(got[got.isinf()], want[want.isinf()])


def test_unused_expert_may_hold_nan():
    T, E, K, F = 30, 4, 64, 64
    shape, lay, recv, _, spans = layout(T, 3, 1, 1, 0, K, 4)
    shape = api.Shape(T, K, E, 1, 1, 0)
    counts = torch.cat([lay.expert_counts, torch.zeros(1, dtype=torch.int32, device="cuda")])
    offsets = torch.cat([lay.expert_offsets, torch.full((1,), T, dtype=torch.int32, device="cuda")])
    lay.expert_counts, lay.expert_offsets = counts, offsets
    w, _ = weights(E, F, K, 4, False)
    w[3] = float("nan")
    y = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    api.moe_expert_matmul(shape, api.Linear(K, F), recv, None, lay, w, None, None, None, y)
    assert not y.isnan().any()


@pytest.mark.parametrize("name,T,E,k,N,C,K,F", [
    ("none", 1, 4, 2, 1, 0, 64, 32),
    ("none", 90, 3, 2, 1, 0, 72, 136),
    ("silu", 40, 6, 2, 2, 30, 104, 48),
    ("gelu", 130, 2, 1, 1, 0, 40, 264),
    ("swiglu", 16, 8, 2, 2, 32, 256, 64),
    ("swiglu", 300, 3, 2, 1, 0, 264, 136),
    ("swiglu", 64, 4, 2, 2, 20, 8, 8),
    ("swiglu", 700, 2, 1, 1, 0, 136, 72),
])
@pytest.mark.parametrize("bad", [False, True])
def test_gradients(name, T, E, k, N, C, K, F, bad, seed=5):
    P = F * (2 if name == "swiglu" else 1)
    shape, lay, recv, _, spans = layout(T, E, k, N, C, K, seed, bad=bad)
    rows = recv.shape[0]
    w, _ = weights(E, P, K, seed, False)
    gen = torch.Generator().manual_seed(seed + 2)
    gy = torch.randn(rows, F, generator=gen).bfloat16().cuda()
    pre = (1.5 * torch.randn(rows, P, generator=gen)).bfloat16().cuda()
    placed = torch.zeros(rows, dtype=torch.bool)
    for a, b in spans:
        placed[a:b] = True
    gy[~placed.cuda()] = float("nan")  # rows of no segment must not matter
    pre[~placed.cuda()] = float("nan")
    full = lambda *s, dt=torch.bfloat16: torch.full(s, FILL, dtype=dt, device="cuda")  # noqa: E731
    gx, gw, gb = full(rows + 2, K), full(E, P, K), full(E, P, dt=torch.float32)
    lin = api.Linear(K, F, ACT[name])
    ws = api.alloc_expert_workspace(shape, lin, "cuda")
    if ws is not None:
        ws.fill_(0xFF)
    z = None if name == "none" else pre
    api.moe_expert_matmul_backward(shape, lin, gy, recv, lay, w, z, gx, gw, gb, ws)
    want, tol = ref.matmul_grad(host(gy), host(recv), host(w), host(pre), spans, name)
    ref.check(gx[:rows], want[0], tol[0], "grad_x", FILL)
    assert (gx[rows:] == FILL).all()
    ref.check(gw, want[1], tol[1], "grad_weight")
    ref.check(gb, want[2], tol[2], "grad_bias")
    # each output alone gives the same
    gx2, gw2, gb2 = full(rows + 2, K), full(E, P, K), full(E, P, dt=torch.float32)
    for out in ((gx2, None, None), (None, gw2, None), (None, None, gb2)):
        api.moe_expert_matmul_backward(shape, lin, gy, recv if out[1] is not None else None, lay,
                                       w if out[0] is not None else None, z, *out, ws)
    assert torch.equal(gx2, gx) and torch.equal(gw2, gw) and torch.equal(gb2, gb)


def test_long_offsets():
    """Rows and elements past 2^31: a segment that starts 2.4e9 elements into x."""
    C, K, F, T = 300000, 8192, 64, 40
    shape = api.Shape(T, K, 2, 1, 2, C)
    x = torch.zeros(2 * C, K, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(T, K, device="cuda").bfloat16()
    x[C:C + T] = rows
    lay = api.Layout.empty(shape, "cuda")
    lay.expert_counts.copy_(torch.tensor([0, T]))
    lay.expert_offsets.copy_(torch.tensor([0, C]))
    w, _ = weights(2, F, K, 1, False)
    y = torch.zeros(2 * C, F, dtype=torch.bfloat16, device="cuda")
    api.moe_expert_matmul(shape, api.Linear(K, F), x, None, lay, w, None, None, None, y)
    want = ref.matmul(host(rows), host(w[1:]), None, None, [(0, T)], "none", F)
    ref.check(y[C:C + T], want[0], want[2], "y")
    assert (y[:C] == 0).all() and (y[C + T:] == 0).all()
    gy = torch.randn(T, F, device="cuda").bfloat16()
    full = torch.zeros(2 * C, F, dtype=torch.bfloat16, device="cuda")
    full[C:C + T] = gy
    gx, gw = torch.zeros_like(x), torch.empty_like(w)
    api.moe_expert_matmul_backward(shape, api.Linear(K, F), full, x, lay, w, None, gx, gw, None)
    grads, tol = ref.matmul_grad(host(gy), host(rows), host(w[1:]), None, [(0, T)], "none")
    ref.check(gx[C:C + T], grads[0], tol[0], "grad_x")
    ref.check(gw[1:], grads[1], tol[1], "grad_weight")
    assert (gw[0] == 0).all()


@pytest.mark.parametrize("name,T,E,k,K,F", [
    ("swiglu", 2100, 2, 1, 72, 11272), ("none", 1030, 1, 1, 128, 22016),
    ("gelu", 900, 3, 2, 200, 16392),
])
def test_many_rows_and_columns(name, T, E, k, K, F):
    """Enough rows per expert and columns for the largest tiles, ragged at both ends."""
    run(T, E, k, 1, 0, K, F, name, seed=T)


@pytest.mark.parametrize("name,T,E,K,F", [("silu", 1100, 2, 16392, 136), ("none", 2050, 4, 8200, 264)])
def test_gradients_of_wide_inputs(name, T, E, K, F):
    shape, lay, recv, _, spans = layout(T, E, 1, 1, 0, K, T)
    w, _ = weights(E, F, K, T, False)
    gen = torch.Generator().manual_seed(T)
    gy = torch.randn(T, F, generator=gen).bfloat16().cuda()
    pre = torch.randn(T, F, generator=gen).bfloat16().cuda()
    gx, gw, gb = torch.empty_like(recv), torch.empty_like(w), torch.empty(E, F, device="cuda")
    lin = api.Linear(K, F, ACT[name])
    z = None if name == "none" else pre
    api.moe_expert_matmul_backward(shape, lin, gy, recv, lay, w, z, gx, gw, gb,
                                   api.alloc_expert_workspace(shape, lin, "cuda"))
    want, tol = ref.matmul_grad(host(gy), host(recv), host(w), host(pre), spans, name)
    for got, wanted, bound, what in zip((gx.view(torch.bfloat16), gw, gb), want, tol,
                                        ("grad_x", "grad_weight", "grad_bias")):
        ref.check(got, wanted, bound, what)


@pytest.mark.parametrize("counts,F,fp8", [
    ([296, 356, 426, 490], 11264, False),      # last tiles of 40, 100, 170, 234 of 256 rows
    ([138, 178, 210, 250, 0], 272, False),     # of 10, 50, 82, 122 of 128
    ([296, 356, 426, 490], 8192, True),
    ([20, 90, 60, 1], 512, True),
])
def test_part_tiles(counts, F, fp8):
    """Every quarter of a tile that the last rows of an expert may reach into."""
    T, E = sum(counts), len(counts)
    K = 128 if fp8 else 72
    run(T, E, 1, 1, 0, K, F, "none", fp8=fp8, counts=counts, seed=T)
    run(T, E, 1, 1, 0, K, F // 2, "swiglu", fp8=fp8, counts=counts, seed=T)


@pytest.mark.parametrize("counts,K", [([296, 356, 426, 490], 11264), ([138, 178, 0, 210, 250], 264)])
def test_part_tiles_of_gradients(counts, K):
    T, E, F = sum(counts), len(counts), 72
    shape, lay, recv, _, spans = layout(T, E, 1, 1, 0, K, T, counts=counts)
    w, _ = weights(E, F, K, T, False)
    gen = torch.Generator().manual_seed(T)
    gy = torch.randn(T, F, generator=gen).bfloat16().cuda()
    gx, gw, gb = torch.empty_like(recv), torch.empty_like(w), torch.empty(E, F, device="cuda")
    lin = api.Linear(K, F)
    api.moe_expert_matmul_backward(shape, lin, gy, recv, lay, w, None, gx, gw, gb,
                                   api.alloc_expert_workspace(shape, lin, "cuda"))
    want, tol = ref.matmul_grad(host(gy), host(recv), host(w), None, spans, "none")
    for got, wanted, bound, what in zip((gx.view(torch.bfloat16), gw, gb), want, tol,
                                        ("grad_x", "grad_weight", "grad_bias")):
        ref.check(got, wanted, bound, what)


@pytest.mark.parametrize("T,E,k", [(100, 200, 4), (9, 1024, 3), (900, 70, 8), (1, 65, 2)])
def test_many_experts(T, E, k):
    """More experts than a wave has lanes, most of them with few rows or none."""
    run(T, E, k, 1, 0, 40, 24, "swiglu", seed=E)
    if E < 1000:
        run(T, E, k, 5 if E % 5 == 0 else 1, 0, 128, 128, "none", fp8=True, seed=E)
    K, F = 40, 24
    shape, lay, recv, _, spans = layout(T, E, k, 1, 0, K, E)
    w, _ = weights(E, F, K, E, False)
    gen = torch.Generator().manual_seed(E)
    gy = torch.randn(T * k, F, generator=gen).bfloat16().cuda()
    gx, gw, gb = torch.empty_like(recv), torch.empty_like(w), torch.empty(E, F, device="cuda")
    lin = api.Linear(K, F)
    api.moe_expert_matmul_backward(shape, lin, gy, recv, lay, w, None, gx, gw, gb,
                                   api.alloc_expert_workspace(shape, lin, "cuda"))
    want, tol = ref.matmul_grad(host(gy), host(recv), host(w), None, spans, "none")
    for got, wanted, bound, what in zip((gx.view(torch.bfloat16), gw, gb), want, tol,
                                        ("grad_x", "grad_weight", "grad_bias")):
        ref.check(got, wanted, bound, what)


def test_no_tokens_with_counts_of_another_batch():
    """No pair can be placed, so no row is looked at, whatever stands in the counts."""
    shape, lin = api.Shape(0, 64, 4, 2, 2, 8), api.Linear(64, 32, 1)
    lay = api.Layout.empty(shape, "cuda")
    lay.expert_counts.fill_(3)
    lay.expert_offsets.copy_(torch.tensor([0, 3, 8, 11]))
    rows = lambda c: torch.full((16, c), FILL, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y, gx, w = rows(32), rows(64), weights(4, 32, 64, 0, False)[0]
    api.moe_expert_matmul(shape, lin, rows(64), None, lay, w, None, None, None, y)
    gw, gb = torch.full_like(w, FILL), torch.full((4, 32), FILL, device="cuda")
    api.moe_expert_matmul_backward(shape, lin, rows(32), rows(64), lay, w, rows(32), gx, gw, gb,
                                   api.alloc_expert_workspace(shape, lin, "cuda"))
    assert (y == FILL).all() and (gx == FILL).all()
    assert (gw == 0).all() and (gb == 0).all()


@pytest.mark.parametrize("S,T,E,k,N,C", [(3, 40, 8, 2, 4, 64), (5, 7, 6, 3, 2, 0), (2, 128, 4, 1, 1, 256)])
def test_rows_of_several_sources(S, T, E, k, N, C):
    """The world's rows after moe_dispatch_sources, and the same through the
    dense rows of the receive half: the same results."""
    H, F = 64, 48
    one = api.Shape(T, H, E, k, N, C)
    world = api.world_shape(one, S)
    gen = torch.Generator().manual_seed(S)
    x = torch.randn(S * T, H, generator=gen).bfloat16().cuda()
    ids = torch.from_numpy(inputs.random_ids(S * T, k, E, 3, distinct=True)).cuda()
    lay = api.Layout.empty(world, "cuda")
    recv, _ = api.alloc_recv(world, "cuda", fill=0xFFFF)
    counts = torch.empty(S, E, dtype=torch.int32, device="cuda")
    api.moe_dispatch_sources(one, S, x, ids, recv, None, lay, counts,
                             torch.empty(E, S, dtype=torch.int32, device="cuda"),
                             api.alloc_workspace(world, "cuda"))
    rows = recv.shape[0]
    w, _ = weights(E, 2 * F, H, 0, False)
    lin = api.Linear(H, F, ACT["swiglu"])
    y = torch.full((rows, F), FILL, dtype=torch.bfloat16, device="cuda")
    api.moe_expert_matmul(world, lin, recv, None, lay, w, None, None, None, y)
    spans = ref.segments(lay.expert_counts.tolist(), lay.expert_offsets.tolist(), E // N, C)
    want = ref.matmul(host(recv), host(w), None, None, spans, "swiglu", F)
    ref.check(y, want[0], want[2], "y", FILL)
    # packed
    dense = api.Shape(S * T, H, E, k, N, 0)
    gx, _ = api.alloc_recv(dense, "cuda", fill=0xFFFF)
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    api.moe_dispatch_recv(world, recv, None, lay, gx, None, off)
    packed = api.Layout.empty(dense, "cuda")
    packed.expert_offsets.copy_(off[:E])
    packed.expert_counts.copy_(off[1:] - off[:E])
    gy = torch.full((S * T * k, F), FILL, dtype=torch.bfloat16, device="cuda")
    api.moe_expert_matmul(dense, lin, gx, None, packed, w, None, None, None, gy)
    for (a, b), o in zip(spans, off.tolist()):
        assert torch.equal(gy[o:o + b - a], y[a:b])


@pytest.mark.parametrize("counts,F", [([2300, 120, 2050], 2816 + 8), ([4100], 4096)])
def test_groups_of_row_tiles(counts, F):
    """More row tiles of an expert than run through together, in equal and in unequal groups."""
    run(sum(counts), len(counts), 1, 1, 0, 64, F, "none", residual=False, pre=False, counts=counts)
