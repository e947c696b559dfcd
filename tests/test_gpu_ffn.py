"""The gated feed-forward block in 8 bits and its gradient against plain fp64 forms:
layouts of dispatch (packed, fixed and overflowing capacity, bad ids, empty and hot
experts), tiles on both sides of every edge, poisoned rows, optional arguments.

Blocks whose second projection is a multiple of the identity show the 8-bit rows
between the projections themselves."""
import pytest
import torch

import expert_reference as ref
import ffn_reference as plain
from combine_moe_dispatch_amd import api, inputs

pytestmark = pytest.mark.gpu

FILL = -7.0
UNIT = 0.875   # 448 codes of a scale 2^-9: exact in 8 bits


def quantized(w):
    """Codes, scales and values of [E, P, K] weights."""
    E, P, K = w.shape
    codes = torch.empty(E, P, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, P // 128, K // 128, device="cuda")
    api.moe_quantize_weight(w.cuda(), codes, scales)
    return codes, scales, ref.widen(codes.cpu(), scales.cpu(), 128)


class Case:
    """Rows dispatched by the library into a poisoned receive buffer, and weights.
    counts: rows of each expert (k == 1)."""

    def __init__(self, T, E, k, N, C, H, I, seed=0, hot=None, bad=False, counts=None, dense=False,
                 up=None, down=None):
        self.shape = api.Shape(T, H, E, k, N, C, 1)
        self.ffn = api.Ffn(H, I)
        gen = torch.Generator().manual_seed(seed)
        x = torch.randn(T, H, generator=gen).bfloat16().cuda()
        if dense:
            self.x, self.xs = torch.empty(T, H, dtype=torch.uint8, device="cuda"), None
            self.xs = torch.empty(T, H // 128, device="cuda")
            api.moe_rms_norm(x, None, torch.ones(H, device="cuda"), 1e-6, None, None, self.x, self.xs)
            self.lay, self.spans = None, [(0, T)]
        else:
            ids = torch.from_numpy(inputs.random_ids(T, k, E, seed, distinct=k <= E, hot=hot)).cuda()
            if counts is not None:
                ids = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).int().cuda()
                ids = ids.view(T, 1)
            if bad:
                ids[::3, 0] = E
                ids[1::5] = -1
            self.lay = api.Layout.empty(self.shape, "cuda")
            self.x, self.xs = api.alloc_recv(self.shape, "cuda", fill=0x7F)  # NaN
            api.moe_dispatch(self.shape, x, ids, self.x, self.xs, self.lay,
                             api.alloc_workspace(self.shape, "cuda"))
            self.spans = ref.segments(self.lay.expert_counts.tolist(),
                                      self.lay.expert_offsets.tolist(), E // N, C)
        self.rows = self.x.shape[0]
        up = torch.randn(E, 2 * I, H, generator=gen) * H ** -0.5 if up is None else up
        down = torch.randn(E, H, I, generator=gen) * I ** -0.5 if down is None else down
        self.up, self.us, self.up64 = quantized(up)
        self.down, self.ds, self.down64 = quantized(down)
        self.x64 = ref.widen(self.x.cpu(), self.xs.cpu(), 1)
        self.gen = gen

    def bf16(self, cols, scale=1.0):
        return (scale * torch.randn(self.rows, cols, generator=self.gen)).bfloat16()

    def out(self, rows, cols):
        return torch.full((rows, cols), FILL, dtype=torch.bfloat16, device="cuda")

    def poisoned(self, backward):
        ws = api.alloc_ffn_workspace(self.shape, self.ffn, "cuda", backward)
        if ws is not None:
            ws.fill_(0xFF)   # NaN codes, NaN floats
        return ws

    def forward(self, residual=None, pre=True, **kw):
        H, I = self.ffn.hidden, self.ffn.intermediate
        y = self.out(self.rows + 3, H)
        z = self.out(self.rows + 3, 2 * I) if pre else None
        api.moe_expert_ffn(self.shape, self.ffn, self.x, self.xs, self.lay, self.up, self.us,
                           self.down, self.ds, residual, y, z, self.poisoned(False), **kw)
        return y, z

    def backward(self, gy, pre, gx=True, gu=True, gd=True, **kw):
        E, H, I = self.shape.num_experts, self.ffn.hidden, self.ffn.intermediate
        gx = self.out(self.rows + 3, H) if gx else None
        gu = self.out(E * 2 * I + 1, H) if gu else None
        gd = self.out(E * H + 1, I) if gd else None
        api.moe_expert_ffn_backward(self.shape, self.ffn, gy, self.x, self.xs, self.lay, self.up,
                                    self.us, self.down, self.ds, pre, gx, gu, gd,
                                    self.poisoned(True), **kw)
        return gx, gu, gd

    def checked_rows(self, most=40):
        """Rows of each expert to compare: all, or the edges of tiles among others."""
        for e, (a, b) in enumerate(self.spans):
            n = b - a
            if n <= most:
                yield e, list(range(a, b))
            else:
                at = {0, 1, 15, 16, 63, 64, 127, 128, 129, 255, 256, n - 17, n - 16, n - 1, n // 2}
                yield e, sorted(a + i for i in at if 0 <= i < n)


def host(t):
    return t.double().cpu()


def check(got, want, bound, what):
    off = (host(got) - want).abs()
    assert (off <= bound).all(), (what, float((off - bound).max()), int((off > bound).sum()))


def check_untouched(case, t):
    placed = torch.zeros(t.shape[0], dtype=torch.bool)
    for a, b in case.spans:
        placed[a:b] = True
    assert (t.cpu()[~placed] == FILL).all(), "a row of no segment was written"


def run_forward(case, residual=True, most=40):
    r = case.bf16(case.ffn.hidden).cuda() if residual else None
    y, z = case.forward(r)
    for e, rows in case.checked_rows(most):
        if not rows:
            continue
        (wy, ty), (wz, tz) = plain.forward(case.x64[rows], case.up64[e], case.down64[e],
                                           None if r is None else host(r)[rows])
        check(z[rows], wz, tz, "pre")
        check(y[rows], wy, ty, "y")
    check_untouched(case, y)
    check_untouched(case, z)


SHAPES = [
    (1, 4, 2, 2, 2, 128, 128),        # one token, fixed capacity
    (1, 1, 1, 1, 0, 640, 128),
    (45, 3, 2, 1, 0, 384, 256),       # packed, odd
    (37, 4, 2, 2, 15, 256, 384),      # capacity overflows
    (200, 2, 1, 2, 150, 128, 640),    # rows nobody reaches
    (600, 3, 2, 1, 0, 256, 128),
]


@pytest.mark.parametrize("T,E,k,N,C,H,I", SHAPES)
def test_forward(T, E, k, N, C, H, I):
    run_forward(Case(T, E, k, N, C, H, I, seed=T))


@pytest.mark.parametrize("T,E,H,I", [(2100, 1, 128, 4096), (1100, 2, 8320, 128), (1300, 3, 256, 3456)])
def test_forward_large_tiles(T, E, H, I):
    """Enough rows and columns for the largest tiles."""
    run_forward(Case(T, E, 1, 1, 0, H, I, seed=T))


@pytest.mark.parametrize("T,E,H,I", [
    (1000, 1, 2048, 2048),    # 256 tiles of 64 rows: whole, one to a compute unit
    (600, 1, 2176, 1792),     # 140 of them
    (1100, 2, 256, 2176),     # 306: tiles of 128 rows
])
def test_forward_flat_tiles(T, E, H, I):
    run_forward(Case(T, E, 1, 1, 0, H, I, seed=T), most=20)


@pytest.mark.parametrize("T,E,k,N,C,H,I,dense", [
    (1, 1, 1, 1, 0, 2048, 128, True),       # the first projection in shares: 8 of 16 steps
    (5, 3, 2, 1, 0, 2176, 256, False),      # 17 steps
    (130, 1, 1, 1, 0, 2048, 2048, True),    # both, and rows of a second tile
    (40, 2, 1, 2, 64, 2048, 128, False),    # rows that nobody reaches
    (70, 80, 3, 8, 500, 2048, 2176, False), # sums lie by placed row: more than 64 experts
    (300, 2, 1, 2, 100, 2304, 128, False),  # capacity overflows
    (3, 40, 1, 1, 0, 2048, 256, False),     # a row an expert, most have none
    (260, 1, 1, 1, 0, 128, 2176, True),     # the second projection alone
])
def test_sums_in_shares(T, E, k, N, C, H, I, dense):
    case = Case(T, E, k, N, C, H, I, seed=T + H, dense=dense)
    run_forward(case, residual=T % 2 == 1, most=10)
    y, z = case.forward()
    for _ in range(3):
        a, b = case.forward()
        assert torch.equal(a, y) and torch.equal(b, z)
    again, _ = case.forward(pre=False)
    assert torch.equal(again, y)


@pytest.mark.parametrize("counts", [
    [1, 0, 2, 16], [17, 0, 0, 15], [63, 64, 65, 0], [127, 128, 129], [255, 256, 257, 1],
    [0, 0, 0, 300], [4] * 30, [191, 192, 193]])
def test_part_tiles(counts):
    E = len(counts)
    case = Case(sum(counts), E, 1, 1, 0, 128, 256, seed=E, counts=counts)
    run_forward(case)
    run_backward(case)


def test_bad_ids_and_hot_expert():
    for kw in (dict(bad=True), dict(hot=1)):
        case = Case(90, 4, 2, 2, 0, 256, 128, seed=3, **kw)
        run_forward(case)
        run_backward(case)


@pytest.mark.parametrize("T", [1, 5, 100, 333])
def test_shared_expert(T):
    """Without a layout, added to a sum in place."""
    case = Case(T, 1, 1, 1, 0, 384, 256, dense=True, seed=T)
    run_forward(case)
    run_backward(case)
    r = case.bf16(384).cuda()
    y, _ = case.forward(r, pre=False)
    api.moe_expert_ffn(case.shape, case.ffn, case.x, case.xs, None, case.up, case.us, case.down,
                       case.ds, r, r)
    assert torch.equal(r, y[:T])


def run_backward(case):
    H, I = case.ffn.hidden, case.ffn.intermediate
    gy, pre = case.bf16(H, 0.01), case.bf16(2 * I)
    gx, gu, gd = case.backward(gy.cuda(), pre.cuda())
    gy64, pre64 = gy.double(), pre.double()
    for e, (a, b) in enumerate(case.spans):
        up, down = gu[e * 2 * I:(e + 1) * 2 * I], gd[e * H:(e + 1) * H]
        if a == b:
            assert (up == 0).all() and (down == 0).all()
            continue
        (wx, tx), (wu, tu), (wd, td) = plain.backward(gy64[a:b], case.x64[a:b], case.up64[e],
                                                      case.down64[e], pre64[a:b])
        check(gx[a:b], wx, tx, "grad_x")
        check(up, wu, tu, "grad_up")
        check(down, wd, td, "grad_down")
    check_untouched(case, gx)
    assert (gu[-1] == FILL).all() and (gd[-1] == FILL).all()
    return gy, pre, gx, gu, gd


@pytest.mark.parametrize("T,E,k,N,C,H,I", SHAPES + [(5, 8, 1, 1, 0, 128, 128)])
def test_backward(T, E, k, N, C, H, I):
    run_backward(Case(T, E, k, N, C, H, I, seed=T + 1))


@pytest.mark.parametrize("T,E,H,I", [(700, 1, 128, 11136), (700, 1, 11136, 128),
                                     (1500, 1, 128, 11136), (1500, 1, 11136, 128)])
def test_backward_large_tiles(T, E, H, I):
    """Enough rows and columns for the larger tiles and for the largest: of the
    activation's slope, of the rows' gradient."""
    case = Case(T, E, 1, 1, 0, H, I, seed=T, dense=True)
    gy, pre = case.bf16(H, 0.01), case.bf16(2 * I)
    gx, gu, gd = case.backward(gy.cuda(), pre.cuda())
    rows = next(case.checked_rows())[1]
    (wx, tx), _, _ = plain.backward(gy.double()[rows], case.x64[rows], case.up64[0],
                                    case.down64[0], pre.double()[rows])
    check(gx[rows], wx, tx, "grad_x")
    check_untouched(case, gx)
    # the weights' gradients, some of their rows: from all token rows
    codes, scales = plain.codes_of(gy.float())
    gq = (codes.unflatten(-1, (-1, 128)) * scales.double()[..., None]).flatten(-2)
    cols = list(range(0, I, max(1, I // 37)))
    gh, dgh = plain.product(gq, torch.zeros_like(gq), case.down64[0][:, cols].T.contiguous())
    g, u = pre.double()[:, cols], pre.double()[:, [I + c for c in cols]]
    s = torch.sigmoid(g)
    x = case.x64
    for at, slope in ((cols, u * s * (1 + g * (1 - s))), ([I + c for c in cols], g * s)):
        gz = gh * slope
        dgz = dgh * slope.abs() + ref.EXP * (gh.abs() + dgh) * (1 + g.abs()) * (1 + u.abs())
        dgz = plain.rounded16(gz, dgz)
        want = gz.T @ x
        bound = (dgz + ref.U16 * (gz.abs() + dgz) + (T + 8) * ref.U32 * gz.abs()).T @ x.abs()
        check(gu[:-1].view(2 * I, H)[at], want, plain.rounded16(want, bound), "grad_up")
    h = g * s * u
    want = gy.double().T @ h
    bound = gy.double().abs().T @ (plain.rounded16(h, ref.EXP * h.abs()) + (T + 8) * ref.U32 * h.abs())
    check(gd[:-1].view(H, I)[:, cols], want, plain.rounded16(want, bound), "grad_down")


@pytest.mark.parametrize("T", [3, 150, 700])
def test_rows_between_the_projections(T):
    """down UNIT times the identity: y shows the 8-bit rows themselves, each as near as
    its code."""
    H = I = 256 if T < 700 else 4096
    eye = UNIT * torch.eye(I)[None]
    case = Case(T, 1, 1, 1, 0, H, I, dense=True, seed=T, down=eye)
    assert torch.equal(case.down64[0], eye[0].double())
    y, _ = case.forward()
    rows = next(case.checked_rows())[1]
    z, dz = plain.product(case.x64[rows], torch.zeros(len(rows), H, dtype=torch.float64), case.up64[0])
    v, slack = plain.quantize(*plain.gated(z, dz))
    v, slack = UNIT * v, UNIT * slack + 2 * ref.U32 * v.abs()
    check(y[rows], v, plain.rounded16(v, slack), "8-bit rows")


@pytest.mark.parametrize("T", [3, 150, 700])
def test_slopes_between_the_projections(T):
    """UNIT times identities: grad_x shows the 8-bit rows of the activation's gradient,
    gate and up half, as their fp32 values round."""
    I = 256 if T < 700 else 4096
    H = 2 * I
    eye = UNIT * torch.eye(H)[None]
    down = torch.zeros(1, H, I)
    down[0, :I] = UNIT * torch.eye(I)     # gh is UNIT times the first half of q(grad_y)
    case = Case(T, 1, 1, 1, 0, H, I, dense=True, seed=T, up=eye, down=down)
    gy, pre = case.bf16(H, 0.01), case.bf16(2 * I)
    gx, _, _ = case.backward(gy.cuda(), pre.cuda(), gu=False, gd=False)
    rows = next(case.checked_rows())[1]
    codes, scales = plain.codes_of(gy.float()[rows])
    gh = UNIT * (codes.unflatten(-1, (-1, 128)) * scales.double()[..., None]).flatten(-2)[:, :I]
    g, u = pre.double()[rows].chunk(2, 1)
    s = torch.sigmoid(g)
    gz = torch.cat([gh * u * s * (1 + g * (1 - s)), gh * g * s], 1)
    d = torch.cat([gh.abs() * u.abs() * s * (1 + g.abs()), gh.abs() * g.abs() * s], 1) * ref.EXP
    v, slack = plain.quantize(gz, d)
    v, slack = UNIT * v, UNIT * slack + 2 * ref.U32 * v.abs()
    check(gx[rows], v, plain.rounded16(v, slack), "8-bit slopes")


def test_optional_arguments():
    case = Case(70, 3, 2, 1, 0, 256, 128, seed=11)
    y, z = case.forward()
    again, none = case.forward(pre=False)
    assert none is None and torch.equal(y, again)
    gy, pre, gx, gu, gd = run_backward(case)
    gy, pre = gy.cuda(), pre.cuda()
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)):
        got = case.backward(gy, pre, *map(bool, want))
        for w, a, b in zip(want, got, (gx, gu, gd)):
            assert torch.equal(a, b) if w else a is None
    # what an output does not need may be left out
    x = api.moe_expert_ffn_backward
    out = torch.empty_like(gd[:-1])
    x(case.shape, case.ffn, gy, None, None, case.lay, None, None, None, None, pre, None, None, out)
    assert torch.equal(out, gd[:-1])


def test_special_values():
    """Rows of zeros, rows with a NaN or an infinity beside rows that keep theirs."""
    case = Case(40, 1, 1, 1, 0, 256, 256, dense=True, seed=2)
    clean, _ = case.forward()
    case.x[3], case.xs[3] = 0, 0.0
    case.x[5, 200] = 0x7F                         # NaN
    case.xs[7, 1] = float("inf")
    y, z = case.forward()
    assert (y[3] == 0).all() and y[5].isnan().all() and y[7].isnan().all()
    rest = [i for i in range(40) if i not in (3, 5, 7)]
    assert torch.equal(y[rest], clean[rest])
    gy, pre = case.bf16(256, 0.01).cuda(), case.bf16(512).cuda()
    gy[4] = 0
    gy[6, 9] = float("nan")
    pre[8, 0] = float("inf")                      # silu'(inf) = 1 - inf * 0
    pre[9, :256] = -1e4                           # a shut gate: no gradient of either half
    gx, _, _ = case.backward(gy, pre, gu=False, gd=False)
    assert (gx[4] == 0).all() and gx[6].isnan().all() and gx[8].isnan().all()
    assert (gx[9] == 0).all()
    assert gx[10:40].isfinite().all()


def test_no_tokens():
    case = Case(4, 2, 1, 1, 0, 128, 128)
    shape = api.Shape(0, 128, 2, 1, 1, 0, 1)
    api.moe_expert_ffn(shape, case.ffn, case.x, case.xs, case.lay, case.up, case.us, case.down,
                       case.ds, None, case.out(0, 128))
    gu, gd = case.out(512, 128), case.out(256, 128)
    api.moe_expert_ffn_backward(shape, case.ffn, case.out(0, 128), None, None, case.lay, None, None,
                                None, None, case.out(0, 256), None, gu, gd)
    assert (gu == 0).all() and (gd == 0).all()


@pytest.mark.parametrize("T,E,k,H,I", [(3, 8, 2, 256, 256), (300, 4, 2, 384, 256)])
def test_repeatable_and_alone(T, E, k, H, I):
    """The same bits again, and whatever rows stand beside an expert's."""
    case = Case(T, E, k, 1, 0, H, I, seed=T)
    y, z = case.forward()
    for _ in range(3):
        a, b = case.forward()
        assert torch.equal(a, y) and torch.equal(b, z)
    gy, pre = case.bf16(H, 0.01).cuda(), case.bf16(2 * I).cuda()
    first = case.backward(gy, pre)
    for _ in range(3):
        for a, b in zip(case.backward(gy, pre), first):
            assert torch.equal(a, b)


def test_refusals_on_tensors():
    case = Case(8, 2, 1, 1, 0, 128, 128)
    y = case.out(8, 128)
    args = [case.shape, case.ffn, case.x, case.xs, case.lay, case.up, case.us, case.down, case.ds,
            None, y, None]

    def call(i, v):
        a = list(args)
        a[i] = v
        api.moe_expert_ffn(*a)

    for i, v, what in ((2, case.x[:4], "x holds"), (3, case.xs[:1], "x_scales holds"),
                       (5, case.up[:1], "up holds"), (6, case.us[:1], "up_scales holds"),
                       (7, case.down[:1], "down holds"), (8, None, "down_scales is required"),
                       (10, y[:2], "y holds"), (9, y[:2], "residual holds"),
                       (11, y, "pre holds")):
        with pytest.raises(ValueError, match=what):
            call(i, v)
    with pytest.raises(TypeError, match="x must be"):
        call(2, case.x.float())
    with pytest.raises(api.MoeError):
        api.moe_expert_ffn(*args, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(api.MoeError):                     # a bf16 payload
        api.moe_expert_ffn(api.Shape(8, 128, 2, 1, 1, 0, 0), *args[1:])


@pytest.mark.parametrize("T,E,k,N,C,H,I,dense", [
    (2, 1, 1, 1, 0, 2048, 2048, True),      # both projections in shares
    (60, 4, 2, 2, 100, 256, 2048, False),   # the second alone, fixed capacity
    (260, 3, 2, 1, 0, 256, 384, False),     # neither
    (2100, 1, 1, 1, 0, 128, 4096, True),    # large tiles
])
def test_residual_in_place(T, E, k, N, C, H, I, dense):
    case = Case(T, E, k, N, C, H, I, seed=T, dense=dense)
    r = case.bf16(H).cuda()
    y, _ = case.forward(r)
    before = r.clone()
    api.moe_expert_ffn(case.shape, case.ffn, case.x, case.xs, case.lay, case.up, case.us, case.down,
                       case.ds, r, r, None, case.poisoned(False))
    placed = torch.zeros(case.rows, dtype=torch.bool, device="cuda")
    for a, b in case.spans:
        placed[a:b] = True
    assert torch.equal(r[placed], y[:case.rows][placed])
    assert torch.equal(r[~placed], before[~placed])
