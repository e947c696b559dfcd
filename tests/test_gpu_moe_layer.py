"""A whole MoE layer's training step through the library: route, dispatch, gate/up
and down projections, combine, a shared expert on top, the balance loss, and back
through all of it; in one HIP graph; on several streams; as a run of single tokens."""
import pytest
import torch

import expert_reference as ref
from combine_moe_dispatch_amd import api

pytestmark = pytest.mark.gpu

COEF = 0.02
DEV = "cuda"


class Layer:
    """Buffers of one layer, as a training program would hold them."""

    def __init__(self, T, H, I, E, k, N, C, score, seed, offsets=None):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        self.T, self.H, self.I, self.E, self.k, self.score = T, H, I, E, k, score
        self.shape = api.Shape(T, H, E, k, N, C)
        self.rows = api.moe_recv_rows(self.shape)
        self.x = r(T, H).bfloat16().to(DEV)
        self.router = (r(E, H) * H ** -0.5).to(DEV)
        self.bias = (0.1 * r(E)).to(DEV)
        self.w1 = (r(E, 2 * I, H) * H ** -0.5).bfloat16().to(DEV)
        self.b1 = (0.1 * r(E, 2 * I)).to(DEV)
        self.w2 = (r(E, H, I) * I ** -0.5).bfloat16().to(DEV)
        self.b2 = (0.1 * r(E, H)).to(DEV)
        self.ws1 = (r(1, I, H) * H ** -0.5).bfloat16().to(DEV)
        self.ws2 = (r(1, H, I) * I ** -0.5).bfloat16().to(DEV)
        self.gout = r(T, H).bfloat16().to(DEV)  # gradient of the layer's output
        self.off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
        S = 1 if offsets is None else len(offsets) - 1
        self.l1 = api.Linear(H, I, api.MOE_ACT_SWIGLU)
        self.l2 = api.Linear(I, H)
        self.s1 = api.Linear(H, I, api.MOE_ACT_GELU)
        self.s2 = api.Linear(I, H)
        self.dense = api.Shape(T, H, 1, 1, 1, 0)
        self.logits = torch.empty(T, E, device=DEV)
        self.ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
        self.w = torch.empty(T, k, device=DEV)
        self.lay = api.Layout.empty(self.shape, DEV)
        self.dws = api.alloc_workspace(self.shape, DEV)
        nan = float("nan")
        self.recv, self.h = bf(self.rows, H).fill_(nan), bf(self.rows, I).fill_(nan)
        self.pre, self.y = bf(self.rows, 2 * I).fill_(nan), bf(self.rows, H).fill_(nan)
        self.routed, self.out = bf(T, H), bf(T, H)
        self.sh, self.spre = bf(T, I), bf(T, I)
        self.counts = torch.empty(S, E, dtype=torch.int32, device=DEV)
        self.probs = torch.empty(S, E, device=DEV)
        self.tokens = torch.empty(S, dtype=torch.int32, device=DEV)
        self.loss = torch.empty(1, device=DEV)
        u8 = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)  # noqa: E731
        self.bws = u8(api.moe_balance_loss_workspace_size(T, E, S))
        self.rws = u8(api.moe_route_backward_workspace_size(T, E))
        self.ws_1 = api.alloc_expert_workspace(self.shape, self.l1, DEV)
        self.ws_2 = api.alloc_expert_workspace(self.shape, self.l2, DEV)
        self.ws_s = api.alloc_expert_workspace(self.dense, self.s1, DEV)
        self.gy, self.gh = bf(self.rows, H), bf(self.rows, I)
        self.grecv, self.gx = bf(self.rows, H), bf(T, H)
        self.gsh, self.gxs = bf(T, I), bf(T, H)
        self.gw = torch.empty(T, k, device=DEV)
        self.ones = torch.ones(T, k, device=DEV)
        self.g = {n: torch.empty_like(getattr(self, n)) for n in
                  ("w1", "b1", "w2", "b2", "ws1", "ws2", "logits", "bias")}

    def forward(self, stream=None):
        s = dict(stream=stream)
        torch.matmul(self.x.float(), self.router.t(), out=self.logits)
        api.moe_route_topk(self.logits, self.bias, self.k, self.score, self.ids, self.w, **s)
        api.moe_balance_loss(self.logits, self.bias, self.ids, self.score, COEF, self.off,
                             self.counts, self.probs, self.tokens, self.loss, self.bws, **s)
        api.moe_dispatch(self.shape, self.x, self.ids, self.recv, None, self.lay, self.dws, **s)
        api.moe_expert_matmul(self.shape, self.l1, self.recv, None, self.lay, self.w1, None,
                              self.b1, None, self.h, self.pre, **s)
        api.moe_expert_matmul(self.shape, self.l2, self.h, None, self.lay, self.w2, None, self.b2,
                              None, self.y, **s)
        api.moe_combine(self.shape, self.y, None, self.lay, self.w, self.routed, **s)
        api.moe_expert_matmul(self.dense, self.s1, self.x, None, None, self.ws1, None, None, None,
                              self.sh, self.spre, **s)
        api.moe_expert_matmul(self.dense, self.s2, self.sh, None, None, self.ws2, None, None,
                              self.routed, self.out, **s)

    def backward(self, stream=None):
        s = dict(stream=stream)
        api.moe_combine_backward(self.shape, self.gout, self.y, self.lay, self.w, self.gy, self.gw,
                                 **s)
        api.moe_expert_matmul_backward(self.shape, self.l2, self.gy, self.h, self.lay, self.w2,
                                       None, self.gh, self.g["w2"], self.g["b2"], self.ws_2, **s)
        api.moe_expert_matmul_backward(self.shape, self.l1, self.gh, self.recv, self.lay, self.w1,
                                       self.pre, self.grecv, self.g["w1"], self.g["b1"], self.ws_1,
                                       **s)
        api.moe_combine(self.shape, self.grecv, None, self.lay, self.ones, self.gx, **s)
        api.moe_expert_matmul_backward(self.dense, self.s2, self.gout, self.sh, None, self.ws2,
                                       None, self.gsh, self.g["ws2"], None, **s)
        api.moe_expert_matmul_backward(self.dense, self.s1, self.gsh, self.x, None, self.ws1,
                                       self.spre, self.gxs, self.g["ws1"], None, self.ws_s, **s)
        api.moe_route_backward(self.logits, self.bias, self.ids, self.w, self.gw, self.score, COEF,
                               self.off, self.counts, self.tokens, None, self.g["logits"],
                               self.g["bias"], workspace=self.rws, **s)

    def results(self):
        out = {"out": self.out, "loss": self.loss, "gx": self.gx, "gxs": self.gxs, **self.g}
        return {n: t.clone() for n, t in out.items()}


class Round(torch.autograd.Function):
    """To bf16 and back, forward and backward: where the library rounds."""

    @staticmethod
    def forward(ctx, t):
        return t.float().bfloat16().double()

    @staticmethod
    def backward(ctx, g):
        return g.float().bfloat16().double()


def reference(L, rounding):
    """The same step in fp64 autograd on the library's routing, with or without
    roundings to bf16 at the library's places."""
    rnd = Round.apply if rounding else (lambda t: t)
    d = lambda t: t.detach().double().cpu().requires_grad_()  # noqa: E731
    p = {n: d(getattr(L, n)) for n in ("w1", "b1", "w2", "b2", "ws1", "ws2", "logits", "bias")}
    xr, xs = d(L.x), d(L.x)  # the routed and the shared branch's input
    ids = L.ids.cpu()
    placed = L.lay.token_row.cpu() >= 0
    biased = p["logits"] + p["bias"]
    w = ref.routed(biased, ids, L.score)
    routed = torch.zeros(L.T, L.H, dtype=torch.float64)
    for e in range(L.E):
        t, j = ((ids == e) & placed).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        z = xr[t] @ p["w1"][e].T + p["b1"][e]
        h = rnd(ref.act("swiglu", z))
        y = rnd(h @ p["w2"][e].T + p["b2"][e])
        routed = routed.index_add(0, t, w[t, j][:, None] * y)
    hs = rnd(ref.act("gelu", xs @ p["ws1"][0].T))
    out = rnd(rnd(routed) + hs @ p["ws2"][0].T)
    off = None if L.off is None else L.off.tolist()
    loss = ref.balance(biased, ids, L.score, off, COEF)[0]
    total = (out * L.gout.double().cpu()).sum() + loss
    names = list(p)
    grads = torch.autograd.grad(total, [p[n] for n in names] + [xr, xs])
    res = dict(zip(names, grads))
    res.update(out=out.detach(), loss=loss.detach().view(1), gx=grads[-2], gxs=grads[-1])
    return res


@pytest.mark.parametrize("T,H,I,E,k,N,C,score,offsets", [
    (70, 128, 72, 6, 2, 2, 0, 0, [0, 30, 70]),
    (64, 256, 64, 8, 2, 2, 24, 1, None),      # capacity overflows
    (300, 136, 96, 4, 3, 1, 0, 1, [0, 1, 150, 290]),
])
def test_training_step(T, H, I, E, k, N, C, score, offsets):
    L = Layer(T, H, I, E, k, N, C, score, T, offsets)
    L.forward()
    L.backward()
    got = L.results()
    exact, rounded = reference(L, False), reference(L, True)
    for n, t in got.items():
        # The library rounds where the reference with roundings does, so its
        # distance from the exact step is that of the roundings: at most twice
        # it, and 2^-18 for fp32 sums where nothing was rounded to bf16.
        size = exact[n].norm()
        off = (t.double().cpu().view(exact[n].shape) - exact[n]).norm()
        own = (rounded[n] - exact[n]).norm()
        assert off <= 2 * own + 2.0 ** -18 * size, (n, float(off / size), float(own / size))


def test_differences():
    """The gradients against central differences of the fp64 step."""
    L = Layer(40, 64, 32, 4, 2, 1, 0, 1, 3)
    L.forward()
    L.backward()
    ids = L.ids.cpu()

    def value(p):
        biased = p["logits"] + p["bias"]
        w = ref.routed(biased, ids, 1)
        out = torch.zeros(L.T, L.H, dtype=torch.float64)
        for e in range(L.E):
            t, j = (ids == e).nonzero(as_tuple=True)
            z = L.x.double().cpu()[t] @ p["w1"][e].T + p["b1"][e]
            y = ref.act("swiglu", z) @ p["w2"][e].T + p["b2"][e]
            out = out.index_add(0, t, w[t, j][:, None] * y)
        hs = ref.act("gelu", L.x.double().cpu() @ p["ws1"][0].T)
        out = out + hs @ p["ws2"][0].T
        return float((out * L.gout.double().cpu()).sum() + ref.balance(biased, ids, 1, None, COEF)[0])

    names = ("w1", "b1", "w2", "b2", "ws1", "ws2", "logits", "bias")
    base = {n: getattr(L, n).double().cpu() for n in names}
    gen = torch.Generator().manual_seed(5)
    h = 1e-5
    for n in names:
        d = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        want = (value({**base, n: base[n] + h * d}) - value({**base, n: base[n] - h * d})) / (2 * h)
        have = float((L.g[n].double().cpu() * d).sum())
        # at most four roundings to bf16 on the way to a term, each off by 2^-8 of
        # it and independent of the others: three times their root sum of squares
        bound = 3 * 4 * ref.U16 * float((L.g[n].double().cpu() * d).norm()) + 1e-6 * abs(want)
        assert abs(want - have) <= bound, (n, want, have)


def test_step_in_a_graph():
    """The whole step captured once and replayed: every replay, with eager work
    and other inputs between them, gives what eager calls give."""
    L = Layer(96, 128, 64, 8, 2, 2, 0, 1, 11, [0, 40, 96])
    other = Layer(96, 128, 64, 8, 2, 2, 0, 1, 12, [0, 40, 96])
    inputs = [(l.x.clone(), l.gout.clone()) for l in (L, other)]
    want = []
    for x, g in inputs:
        L.x.copy_(x)
        L.gout.copy_(g)
        L.forward()
        L.backward()
        torch.cuda.synchronize()
        want.append(L.results())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.forward()
        L.backward()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward()
        L.backward()
    for i in (0, 1, 0, 1):
        L.x.copy_(inputs[i][0])
        L.gout.copy_(inputs[i][1])
        for t in (L.h, L.pre, L.y, L.gy, L.gh, L.grecv, *L.g.values()):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        other.forward()  # eager work between the replays
        torch.cuda.synchronize()
        for n, t in L.results().items():
            assert torch.equal(t, want[i][n]), n


def test_streams_at_once():
    """Four layers on four streams at once equal the same layers one by one."""
    sizes = [(96, 128, 64, 8, 2, 2, 0, 1), (300, 64, 48, 4, 1, 1, 0, 0), (1, 256, 72, 8, 4, 2, 8, 1),
             (513, 72, 40, 3, 2, 1, 0, 0)]
    alone = []
    for i, s in enumerate(sizes):
        L = Layer(*s, seed=i)
        L.forward()
        L.backward()
        torch.cuda.synchronize()
        alone.append(L.results())
    layers = [Layer(*s, seed=i) for i, s in enumerate(sizes)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    for _ in range(2):
        for L, st in zip(layers, streams):
            with torch.cuda.stream(st):
                L.forward()
                L.backward()
    torch.cuda.synchronize()
    for L, want in zip(layers, alone):
        for n, t in L.results().items():
            assert torch.equal(t, want[n]), n


def test_given_stream_and_own_workspaces():
    """Calls given a stream, which allocate their workspaces themselves."""
    T, E, k = 500, 64, 4
    l = torch.randn(T, E, device=DEV)
    ids, w = api.moe_route_topk(l, None, k, 1)
    gw = torch.randn(T, k, device=DEV)
    want = api.moe_balance_loss(l, None, ids, 1, COEF)
    want_g = api.moe_route_backward(l, None, ids, w, gw, 1, COEF, None, want[1], want[3],
                                    with_grad_bias=True)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for given in (st, st.cuda_stream):
        got = api.moe_balance_loss(l, None, ids, 1, COEF, stream=given)
        st.synchronize()
        g = api.moe_route_backward(l, None, ids, w, gw, 1, COEF, None, got[1], got[3],
                                   with_grad_bias=True, stream=given)
        st.synchronize()
        for a, b in zip((*got, *g), (*want, *want_g)):
            assert torch.equal(a, b)


def test_tokens_one_by_one_equal_the_batch():
    """Rows do not depend on their neighbours: single-token calls give the
    batch's values within the bound of either's sums."""
    T, H, I, E, k = 6, 192, 80, 8, 2
    L = Layer(T, H, I, E, k, 1, 0, 1, 21)
    L.forward()
    rows = L.lay.token_row.cpu()
    x64, w64 = L.x.double().cpu(), L.w1.double().cpu()
    for t in range(T):
        one = api.Shape(1, H, E, k, 1, 0)
        lay = api.Layout.empty(one, DEV)
        recv = torch.empty(k, H, dtype=torch.bfloat16, device=DEV)
        api.moe_dispatch(one, L.x[t:t + 1], L.ids[t:t + 1], recv, None, lay)
        h = torch.empty(k, I, dtype=torch.bfloat16, device=DEV)
        api.moe_expert_matmul(one, L.l1, recv, None, lay, L.w1, None, L.b1, None, h)
        for j in range(k):
            e = int(L.ids[t, j])
            want, _, tol, _ = ref.matmul(x64[t:t + 1], w64[e:e + 1], L.b1[e:e + 1].double().cpu(),
                                         None, [(0, 1)], "swiglu", I)
            got = h[int(lay.token_row[0, j])].double().cpu()
            batch = L.h[int(rows[t, j])].double().cpu()
            assert ((got - want[0]).abs() <= tol[0]).all()
            assert ((batch - want[0]).abs() <= tol[0]).all()
