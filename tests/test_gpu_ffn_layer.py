"""An expert layer in 8 bits through the library: norm, route, dispatch, experts and a
shared expert, combine, the next layer's norm, and back through all of it; against
fp64 without any rounding; in one HIP graph; on given streams at once; and sizes past
32 bits."""
import subprocess
import sys

import pytest
import torch

import expert_reference as ref
import ffn_reference as plain
from combine_moe_dispatch_amd import api

pytestmark = pytest.mark.gpu

EPS = 1e-6
DEV = "cuda"


class Layer:
    """Buffers of one layer, as a training program would hold them."""

    def __init__(self, T, H, I, E, k, N, C, seed):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
        f32 = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
        self.T, self.k = T, k
        self.shape = api.Shape(T, H, E, k, N, C, api.MOE_PAYLOAD_FP8_E4M3_B128)
        self.back = api.Shape(T, H, E, k, N, C)           # the way back is bf16
        self.dense = api.Shape(T, H, 1, 1, 1, 0, api.MOE_PAYLOAD_FP8_E4M3_B128)
        self.ffn = api.Ffn(H, I)
        rows = api.moe_recv_rows(self.shape)
        self.x, self.res = r(T, H).bfloat16().to(DEV), r(T, H).bfloat16().to(DEV)
        self.nw, self.nw2 = (1 + 0.1 * r(H)).to(DEV), (1 + 0.1 * r(H)).to(DEV)
        self.router = (r(E, H) * H ** -0.5).to(DEV)
        # master weights: fp32 for the experts, bf16 for the shared one
        self.up, self.down = (r(E, 2 * I, H) * H ** -0.5).to(DEV), (r(E, H, I) * I ** -0.5).to(DEV)
        self.sup = (r(1, 2 * I, H) * H ** -0.5).bfloat16().to(DEV)
        self.sdown = (r(1, H, I) * I ** -0.5).bfloat16().to(DEV)
        self.codes = {}
        for n in ("up", "down", "sup", "sdown"):
            w = getattr(self, n)
            self.codes[n] = u8(w.shape), f32(w.shape[0], w.shape[1] // 128, w.shape[2] // 128)
        self.gout = (0.1 * r(T, H)).bfloat16().to(DEV)
        self.total, self.y, self.q, self.qs, self.inv = bf(T, H), bf(T, H), u8(T, H), f32(T, H // 128), f32(T)
        self.logits, self.ids = f32(T, E), torch.empty(T, k, dtype=torch.int32, device=DEV)
        self.w, self.gw, self.ones = f32(T, k), f32(T, k), torch.ones(T, k, device=DEV)
        self.lay = api.Layout.empty(self.shape, DEV)
        self.dws = api.alloc_workspace(self.shape, DEV)
        self.recv, self.rs = api.alloc_recv(self.shape, DEV, fill=0x7F)
        self.ey, self.pre = bf(rows, H), bf(rows, 2 * I)
        self.routed, self.out, self.spre = bf(T, H), bf(T, H), bf(T, 2 * I)
        self.total2, self.y2, self.inv2 = bf(T, H), bf(T, H), f32(T)
        self.ws, self.dws_s = (api.alloc_ffn_workspace(s, self.ffn, DEV) for s in (self.shape, self.dense))
        self.bws, self.bws_s = (api.alloc_ffn_workspace(s, self.ffn, DEV, backward=True)
                                for s in (self.shape, self.dense))
        self.nws = api.alloc_rms_norm_workspace(T, H, DEV)
        self.gtotal2, self.gey, self.grecv = bf(T, H), bf(rows, H), bf(rows, H)
        self.gx, self.gxs, self.gy, self.gin = bf(T, H), bf(T, H), bf(T, H), bf(T, H)
        self.gnw, self.gnw2 = f32(H), f32(H)
        self.g = {n: bf(*getattr(self, n).shape) for n in ("up", "down", "sup", "sdown")}

    def forward(self, stream=None):
        s = dict(stream=stream)
        for n, (c, sc) in self.codes.items():
            api.moe_quantize_weight(getattr(self, n), c, sc, **s)
        api.moe_rms_norm(self.x, self.res, self.nw, EPS, self.total, self.y, self.q, self.qs, self.inv,
                         **s)
        torch.matmul(self.y.float(), self.router.t(), out=self.logits)
        api.moe_route_topk(self.logits, None, self.k, api.MOE_SCORE_SIGMOID, self.ids, self.w, **s)
        api.moe_dispatch(self.shape, self.y, self.ids, self.recv, self.rs, self.lay, self.dws, **s)
        api.moe_expert_ffn(self.shape, self.ffn, self.recv, self.rs, self.lay, *self.codes["up"],
                           *self.codes["down"], None, self.ey, self.pre, self.ws, **s)
        api.moe_combine(self.back, self.ey, None, self.lay, self.w, self.routed, **s)
        api.moe_expert_ffn(self.dense, self.ffn, self.q, self.qs, None, *self.codes["sup"],
                           *self.codes["sdown"], self.routed, self.out, self.spre, self.dws_s, **s)
        api.moe_rms_norm(self.out, self.total, self.nw2, EPS, self.total2, self.y2, None, None,
                         self.inv2, **s)

    def backward(self, stream=None):
        """From the gradient of y2; the routed weights' own gradient stops at gw."""
        s = dict(stream=stream)
        api.moe_rms_norm_backward(self.gout, self.total2, self.nw2, self.inv2, None, self.gtotal2,
                                  self.gnw2, self.nws, **s)
        api.moe_combine_backward(self.back, self.gtotal2, self.ey, self.lay, self.w, self.gey, self.gw,
                                 **s)
        api.moe_expert_ffn_backward(self.shape, self.ffn, self.gey, self.recv, self.rs, self.lay,
                                    *self.codes["up"], *self.codes["down"], self.pre, self.grecv,
                                    self.g["up"], self.g["down"], self.bws, **s)
        api.moe_combine(self.back, self.grecv, None, self.lay, self.ones, self.gx, **s)
        api.moe_expert_ffn_backward(self.dense, self.ffn, self.gtotal2, self.q, self.qs, None,
                                    *self.codes["sup"], *self.codes["sdown"], self.spre, self.gxs,
                                    self.g["sup"], self.g["sdown"], self.bws_s, **s)
        torch.add(self.gx, self.gxs, out=self.gy)
        api.moe_rms_norm_backward(self.gy, self.total, self.nw, self.inv, self.gtotal2, self.gin,
                                  self.gnw, self.nws, **s)

    def results(self):
        out = {"y2": self.y2, "total2": self.total2, "gin": self.gin, "gnw": self.gnw,
               "gnw2": self.gnw2, "gw": self.gw, **self.g}
        return {n: t.clone() for n, t in out.items()}

    def exact(self):
        """The same layer in fp64 autograd without any rounding, for the library's ids."""
        d = lambda t: t.double().cpu().requires_grad_()  # noqa: E731
        x, nw, nw2 = d(self.x.float() + self.res.float()), d(self.nw), d(self.nw2)
        up, down, sup, sdown = d(self.up), d(self.down), d(self.sup), d(self.sdown)
        norm = lambda t, w: t * (t.square().mean(1, keepdim=True) + EPS).rsqrt() * w  # noqa: E731
        block = lambda t, u, v: ref.act("swiglu", t @ u.T) @ v.T  # noqa: E731
        y = norm(x, nw)
        w = self.w.double().cpu().requires_grad_()
        out = block(y, sup[0], sdown[0])
        for e in range(up.shape[0]):
            t, j = (self.ids.cpu() == e).nonzero(as_tuple=True)
            out = out.index_add(0, t, w[t, j, None] * block(y[t], up[e], down[e]))
        total2 = x + out
        y2 = norm(total2, nw2)
        leaves = dict(gin=x, gnw=nw, gnw2=nw2, gw=w, up=up, down=down, sup=sup, sdown=sdown)
        grads = torch.autograd.grad((y2 * self.gout.double().cpu()).sum(), list(leaves.values()))
        return {"y2": y2.detach(), "total2": total2.detach(), **dict(zip(leaves, grads))}


# An e4m3 rounding is off by 2^-4 / sqrt 3 of the value at most on average: 3.6%.  A
# product of two rounded operands 5.1%; the activation's factors both have that, at
# slopes of at most 1.13, and h is rounded: 8.9%; with the second weights 9.6%.  A
# rows' gradient passes grad_y (3.6%) and a weight (3.6%), slopes made of z (two factors
# of 5.1% x 1.13), a rounding and another weight: 11%.  The weights' gradients have
# fewer.  All of it in the 2-norm, errors taken as independent; half as much again.
LOSS = 0.165


@pytest.mark.parametrize("T,H,I,E,k,N,C", [(1, 256, 128, 4, 2, 1, 0), (70, 384, 256, 6, 2, 2, 140),
                                           (300, 512, 384, 4, 3, 1, 0)])
def test_layer_against_exact(T, H, I, E, k, N, C):
    layer = Layer(T, H, I, E, k, N, C, seed=T)
    layer.forward()
    layer.backward()
    got, want = layer.results(), layer.exact()
    # a routed weight's gradient is <g, y>, some 1 / sqrt H of |g| |y| for directions
    # that have nothing to do with each other: an error of y, a share of |y| in any
    # direction, is that share of |g| |y| and no share of the product
    g, y = layer.gtotal2.double().cpu(), layer.ey.double().cpu()
    size = g.norm(dim=1, keepdim=True) * y.norm(dim=1)[layer.lay.token_row.cpu().long()]
    assert ((got.pop("gw").double().cpu() - want.pop("gw")).abs() <= LOSS * size).all()
    for n, w in want.items():
        off = float((got[n].double().cpu() - w).norm() / w.norm())
        print(n, off)
        assert off <= LOSS, (n, off)


def test_the_dispatch_and_the_norm_round_alike():
    """Codes of moe_dispatch from y and codes that the norm makes beside y: the same
    values but for the rounding of y to bf16."""
    layer = Layer(50, 256, 128, 1, 1, 1, 0, seed=3)
    layer.forward()
    a = ref.widen(layer.recv.cpu(), layer.rs.cpu(), 1)
    b = ref.widen(layer.q.cpu(), layer.qs.cpu(), 1)
    y = layer.y.double().cpu()
    step = 2.0 ** -4 * y.abs() + 2.0 ** -10 * layer.qs.double().cpu().repeat_interleave(128, 1)
    assert ((a - y).abs() <= step * 1.01).all()
    assert ((b - y).abs() <= step * 1.01 + ref.U16 * y.abs()).all()


@pytest.mark.parametrize("T", [2, 200])
def test_layer_in_a_graph(T):
    """Captured once, replayed with other inputs, with eager work between: every
    replay gives the eager results."""
    layer = Layer(T, 256, 256, 4, 2, 2, 2 * T, seed=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward()
        layer.backward()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward()
        layer.backward()
    other = Layer(T, 256, 256, 4, 2, 2, 2 * T, seed=5)
    for i in range(4):
        gen = torch.Generator().manual_seed(i)
        x = torch.randn(T, 256, generator=gen).bfloat16()
        up = torch.randn(4, 512, 256, generator=gen) / 16
        for one in (layer, other):
            one.x.copy_(x)
            one.up.copy_(up)
        for ws in (layer.ws, layer.dws_s, layer.bws, layer.bws_s, layer.nws):
            if ws is not None:
                ws.fill_(0xFF)
        graph.replay()
        other.forward()
        other.backward()
        torch.cuda.synchronize()
        for (n, a), b in zip(layer.results().items(), other.results().values()):
            assert torch.equal(a, b), (i, n)


def test_layers_on_streams_at_once():
    """Three layers on streams of their own, queued without waiting, and the calls
    given their stream by hand."""
    def make(i):
        return Layer(120 + 40 * i, 256, 128, 4, 2, 1, 0, seed=20 + i)

    alone = []
    for i in range(3):
        layer = make(i)
        layer.forward()
        layer.backward()
        alone.append(layer.results())
    layers, streams = [make(i) for i in range(3)], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(3):
        for layer, s in zip(layers, streams):
            with torch.cuda.stream(s):  # torch's own products between the calls
                layer.forward(stream=s)
                layer.backward(stream=s)
    torch.cuda.synchronize()
    for layer, want in zip(layers, alone):
        for (n, a), b in zip(layer.results().items(), want.values()):
            assert torch.equal(a, b), n


def test_workspaces_of_their_own():
    """Calls that get no workspace take one for themselves, from their stream's pool."""
    layer = Layer(60, 256, 128, 4, 2, 1, 0, seed=8)
    layer.forward()
    layer.backward()
    want = layer.results()
    layer.ws = layer.dws_s = layer.bws = layer.bws_s = layer.nws = None
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(3):
            layer.forward(stream=s)
            layer.backward(stream=s)
    torch.cuda.synchronize()
    for (n, a), b in zip(layer.results().items(), want.values()):
        assert torch.equal(a, b), n


def test_weights_past_2_31_bytes():
    """The last of 80 experts, whose weights and gradients lie past 32-bit offsets."""
    E, H, I, T = 80, 7168, 2048, 3
    shape, f = api.Shape(T, H, E, 1, 1, 0, 1), api.Ffn(H, I)
    gen = torch.Generator().manual_seed(1)
    up = torch.zeros(E, 2 * I, H, dtype=torch.uint8, device=DEV)
    down = torch.zeros(E, H, I, dtype=torch.uint8, device=DEV)
    us = torch.zeros(E, 2 * I // 128, H // 128, device=DEV)
    ds = torch.zeros(E, H // 128, I // 128, device=DEV)
    w = (torch.randn(2 * I, H, generator=gen) * H ** -0.5).to(DEV)
    v = (torch.randn(H, I, generator=gen) * I ** -0.5).to(DEV)
    api.moe_quantize_weight(w, up[-1], us[-1])
    api.moe_quantize_weight(v, down[-1], ds[-1])
    x = torch.randn(T, H, generator=gen).to(DEV).bfloat16()
    ids = torch.full((T, 1), E - 1, dtype=torch.int32, device=DEV)
    lay = api.Layout.empty(shape, DEV)
    recv, rs = api.alloc_recv(shape, DEV)
    api.moe_dispatch(shape, x, ids, recv, rs, lay, api.alloc_workspace(shape, DEV))
    y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    pre = torch.empty(T, 2 * I, dtype=torch.bfloat16, device=DEV)
    api.moe_expert_ffn(shape, f, recv, rs, lay, up, us, down, ds, None, y, pre)
    x64 = ref.widen(recv.cpu(), rs.cpu(), 1)
    up64, down64 = ref.widen(up[-1].cpu(), us[-1].cpu(), 128), ref.widen(down[-1].cpu(), ds[-1].cpu(), 128)
    (wy, ty), (wz, tz) = plain.forward(x64, up64, down64, None)
    assert ((pre.double().cpu() - wz).abs() <= tz).all()
    assert ((y.double().cpu() - wy).abs() <= ty).all()
    gy = (0.01 * torch.randn(T, H, generator=gen)).bfloat16()
    gx = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    gu = torch.empty(E, 2 * I, H, dtype=torch.bfloat16, device=DEV)
    gd = torch.empty(E, H, I, dtype=torch.bfloat16, device=DEV)
    api.moe_expert_ffn_backward(shape, f, gy.to(DEV), recv, rs, lay, up, us, down, ds, pre, gx, gu, gd)
    grads = plain.backward(gy.double(), x64, up64, down64, pre.double().cpu())
    for got, (want, bound), n in zip((gx, gu[-1], gd[-1]), grads, ("grad_x", "grad_up", "grad_down")):
        assert ((got.double().cpu() - want).abs() <= bound).all(), n
    assert not gu[:-1].any() and not gd[:-1].any()


def test_rows_past_2_31_elements():
    """The last rows of 300001, whose columns lie past 32-bit offsets."""
    T, H, I = 300001, 7168, 128
    shape, f = api.Shape(T, H, 1, 1, 1, 0, 1), api.Ffn(H, I)
    gen = torch.Generator().manual_seed(2)
    codes = {}
    for n, (P, K) in dict(up=(2 * I, H), down=(H, I)).items():
        w = (torch.randn(P, K, generator=gen) * K ** -0.5).to(DEV)
        codes[n] = (torch.empty(P, K, dtype=torch.uint8, device=DEV),
                    torch.empty(P // 128, K // 128, device=DEV))
        api.moe_quantize_weight(w, *codes[n])
    at = [0, 149797, 299593, 299776, 300000]
    x = torch.zeros(T, H, dtype=torch.uint8, device=DEV)
    xs = torch.ones(T, H // 128, device=DEV)
    some = torch.randint(0, 100, (len(at), H), generator=gen).to(torch.uint8)
    x[at], xs[at] = some.to(DEV), 0.01
    y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    pre = torch.empty(T, 2 * I, dtype=torch.bfloat16, device=DEV)
    api.moe_expert_ffn(shape, f, x, xs, None, *codes["up"], *codes["down"], None, y, pre)
    x64 = ref.widen(some, xs[at].cpu(), 1)
    up64, down64 = (ref.widen(c.cpu(), s.cpu(), 128) for c, s in codes.values())
    (wy, ty), (wz, tz) = plain.forward(x64, up64, down64, None)
    assert ((pre[at].double().cpu() - wz).abs() <= tz).all()
    assert ((y[at].double().cpu() - wy).abs() <= ty).all()
    assert not y[1:149797].any()
    gy = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    gsome = (0.01 * torch.randn(len(at), H, generator=gen)).bfloat16()
    gy[at] = gsome.to(DEV)
    gx = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    gu = torch.empty(2 * I, H, dtype=torch.bfloat16, device=DEV)
    gd = torch.empty(H, I, dtype=torch.bfloat16, device=DEV)
    api.moe_expert_ffn_backward(shape, f, gy, x, xs, None, *codes["up"], *codes["down"], pre, gx, gu, gd)
    grads = plain.backward(gsome.double(), x64, up64, down64, pre[at].double().cpu())
    # the other rows are zeros and add nothing to the sums
    for got, (want, bound), n in zip((gx[at], gu, gd), grads, ("grad_x", "grad_up", "grad_down")):
        assert ((got.double().cpu() - want).abs() <= bound).all(), n


@pytest.mark.parametrize("T,H,I,E,k,N,C", [(1, 256, 128, 4, 2, 1, 0), (70, 384, 256, 6, 2, 2, 140),
                                           (300, 512, 384, 4, 3, 1, 0)])
def test_gradient_of_the_routed_weights(T, H, I, E, k, N, C):
    """<g, y> of the layer's own gradient and expert rows, as near as its fp32 sum."""
    layer = Layer(T, H, I, E, k, N, C, seed=T)
    layer.forward()
    layer.backward()
    g, y = layer.gtotal2.double().cpu(), layer.ey.double().cpu()
    terms = g[:, None] * y[layer.lay.token_row.cpu().long().view(T, k)]
    want, bound = terms.sum(2), (H + 8) * ref.U32 * terms.abs().sum(2)
    assert ((layer.gw.double().cpu() - want).abs() <= bound).all()
    assert want.norm() > 100 * bound.norm()   # zeros, or another sign, would not do


def test_two_graphs_at_once():
    """Two layers captured with buffers and workspaces of their own, replayed on two
    streams at the same time with eager work in between."""
    def make(i):
        return Layer(150 + 60 * i, 256, 128, 4, 2, 1, 0, seed=40 + i)

    alone = [make(i) for i in range(2)]
    layers, streams = [make(i) for i in range(2)], [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for layer, s in zip(layers, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            layer.forward()
            layer.backward()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            layer.forward()
            layer.backward()
    for i in range(4):
        for a, b in zip(layers, alone):
            x = torch.randn(a.x.shape, generator=torch.Generator().manual_seed(i)).bfloat16()
            for one in (a, b):
                one.x.copy_(x)
            for ws in (a.ws, a.dws_s, a.bws, a.bws_s, a.nws):
                if ws is not None:
                    ws.fill_(0xFF)
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(layers, alone)):
            b.forward()
            b.backward()
            for (name, got), want in zip(a.results().items(), b.results().values()):
                assert torch.equal(got, want), (i, n, name)


FIRST = """
import sys, torch
sys.path.insert(0, ".")
from combine_moe_dispatch_amd import api
T, H, I = {T}, {H}, {I}
u8 = lambda *s: torch.randint(0, 100, s, dtype=torch.uint8, device="cuda")
f32 = lambda *s: torch.rand(*s, device="cuda") * 1e-3
bf = lambda *s: torch.randn(*s, device="cuda").bfloat16()
x, xs, w = u8(T, H), f32(T, H // 128), (u8(1, 2 * I, H), f32(1, 2 * I // 128, H // 128),
                                        u8(1, H, I), f32(1, H // 128, I // 128))
up, codes, scales = bf(1, 2 * I, H), u8(1, 2 * I, H), f32(1, 2 * I // 128, H // 128)
t, nw, y, pre, gy = bf(T, H), 1 + f32(H), bf(T, H), bf(T, 2 * I), bf(T, H)
gx, gu, gd, n, inv, gn, gw = bf(T, H), bf(1, 2 * I, H), bf(1, H, I), bf(T, H), f32(T), bf(T, H), f32(H)
s, f = api.Shape(T, H, 1, 1, 1, 0, 1), api.Ffn(H, I)
ws, bws = (api.alloc_ffn_workspace(s, f, "cuda", b) for b in (False, True))
nws = api.alloc_rms_norm_workspace(T, H, "cuda")
outs = (codes, scales, y, pre, gx, gu, gd, n, inv, gn, gw)
torch.cuda.synchronize()
def step():
    api.moe_quantize_weight(up, codes, scales)
    api.moe_expert_ffn(s, f, x, xs, None, *w, None, y, pre, ws)
    api.moe_expert_ffn_backward(s, f, gy, x, xs, None, *w, pre, gx, gu, gd, bws)
    api.moe_rms_norm(t, None, nw, 1e-6, None, n, None, None, inv)
    api.moe_rms_norm_backward(gy, t, nw, inv, None, gn, gw, nws)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
for _ in range(3):
    for o in outs:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    step()
    torch.cuda.synchronize()
    for a, b in zip(got, outs):
        assert torch.equal(a, b) and a.any()
print("captured ok")
"""


@pytest.mark.parametrize("T,H,I", [(3, 2048, 2048), (300, 256, 384), (1500, 128, 11136)])
def test_first_calls_inside_a_capture(T, H, I):
    """A process whose first calls of these kernels are captured ones: in shares, and on
    smaller and larger tiles."""
    r = subprocess.run([sys.executable, "-c", FIRST.format(T=T, H=H, I=I)], capture_output=True,
                       text=True, timeout=100)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stderr[-2000:]
