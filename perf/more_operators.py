"""The operators of an expert layer in 8 bits, as cases that can be timed.

Operators: the RMS norm in front of the layer, with the residual's addition
and rows in 8 bits; that norm's gradient; 8-bit weights from the master
weights; the gated feed-forward block of the experts, both projections with
the activation and the 8-bit rows between them; and that block's gradient.

8-bit rows are e4m3 codes with one fp32 scale per 128 neighbouring columns
(weights: per 128 x 128 block): scale = largest magnitude / 448, code =
e4m3(value / scale), both divisions in fp32, zeros where the scale is 0.

`run` computes a case in its plain form, elementary torch operations in fp32
rounded once where the operator rounds, or with `own` set through this
library's calls.  `exact` gives the same results in fp64, from the definitions.

Receive rows are packed: expert segments back to back in expert order, inside
a segment the (token, slot) pairs ascending.  A padded token has no expert
(all its ids are -1) and its pairs have no row.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of a decode step: the norm's latency, rows for the router and the shared expert
        {"name": "norm_token", "op": "norm", "T": 1, "H": 7168, "residual": True, "y": True,
         "codes": True, "save": False},
        # a prefill or training batch, what the backward pass needs kept
        {"name": "norm_prefill", "op": "norm", "T": 4096, "H": 7168, "residual": True, "y": True,
         "codes": True, "save": True},
        # the norm's gradient of a small layer, odd sizes, nothing carried past the norm
        {"name": "norm_grad_small", "op": "norm_grad", "T": 301, "H": 1432, "carried": False},
        # and of a long training batch, with the residual stream's own gradient
        {"name": "norm_grad_long", "op": "norm_grad", "T": 16384, "H": 7168, "carried": True},
        # a shared expert's down projection after an update, bf16 master weights
        {"name": "weights_shared", "op": "weights", "E": 1, "P": 7168, "K": 2048, "type": "bf16"},
        # the gate/up projections of one rank's experts, fp32 master weights
        {"name": "weights_experts", "op": "weights", "E": 32, "P": 4096, "K": 7168,
         "type": "fp32"},
        # one token: eight experts' weights are streamed
        {"name": "ffn_token", "op": "ffn", "T": 1, "E": 32, "k": 8, "H": 7168, "I": 2048,
         "residual": False, "save": False, "padded": False},
        # a decode batch
        {"name": "ffn_decode", "op": "ffn", "T": 128, "E": 32, "k": 8, "H": 7168, "I": 2048,
         "residual": False, "save": False, "padded": False},
        # the shared expert, added to the routed sum, odd token count
        {"name": "ffn_shared", "op": "ffn", "T": 1021, "E": 1, "k": 1, "H": 7168, "I": 2048,
         "residual": True, "save": False, "padded": False},
        # a prefill or training batch, pre-activations kept for the backward pass
        {"name": "ffn_prefill", "op": "ffn", "T": 4096, "E": 32, "k": 8, "H": 7168, "I": 2048,
         "residual": False, "save": True, "padded": True},
        # gradients of a small layer, odd token count
        {"name": "ffn_grad_small", "op": "ffn_grad", "T": 301, "E": 6, "k": 2, "H": 640, "I": 384,
         "padded": True},
        # gradients of one rank's experts for a training micro-batch
        {"name": "ffn_grad", "op": "ffn_grad", "T": 2048, "E": 32, "k": 8, "H": 7168, "I": 2048,
         "padded": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "weights", "ffn", "ffn", "ffn", "ffn_grad"])
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op == "norm":
        codes = yes()
        H = 128 * _log_int(rng, 1, 64) if codes else 8 * _log_int(rng, 8, 1024)
        return {"op": op, "T": _log_int(rng, 1, 16384), "H": H, "residual": yes(),
                "y": not codes or yes(), "codes": codes, "save": yes()}
    if op == "norm_grad":
        return {"op": op, "T": _log_int(rng, 1, 16384), "H": 8 * _log_int(rng, 8, 1024),
                "carried": yes()}
    if op == "weights":
        return {"op": op, "E": _log_int(rng, 1, 32), "P": 128 * _log_int(rng, 1, 32),
                "K": 128 * _log_int(rng, 1, 56), "type": rng.choice(["bf16", "fp32"])}
    E = rng.choice([1, rng.randint(2, 32), rng.randint(8, 32)])
    case = {"op": op, "T": 0, "E": E, "k": rng.randint(1, min(E, 8)),
            "H": 128 * _log_int(rng, 1, 56), "I": 128 * _log_int(rng, 1, 16)}
    if op == "ffn":
        return {**case, "T": _log_int(rng, 1, 4096), "residual": yes(), "save": yes(),
                "padded": yes()}
    return {**case, "T": _log_int(rng, 1, 2048), "padded": yes()}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _blocks(t, rows, cols):
    """e4m3 codes and fp32 scales of a [..., R, C] tensor in blocks of rows x cols."""
    R, C = t.shape[-2], t.shape[-1]
    b = t.view(*t.shape[:-2], R // rows, rows, C // cols, cols)
    scale = b.abs().amax(dim=(-3, -1))
    scale = scale / torch.full_like(scale, 448.0)  # by a number it would be times 1/448
    s = scale[..., :, None, :, None]
    codes = torch.where(s > 0, b / s, 0.0)
    return codes.reshape(t.shape).to(E4M3), scale.contiguous()


def _route(case, gen):
    """Packed layout of a random routing: counts, offsets, row of each pair."""
    T, E, k = case["T"], case["E"], case["k"]
    ids = torch.topk(torch.randn(T, E, generator=gen, device=DEVICE), k, dim=1).indices
    if case["padded"]:  # about one token in eleven, never all
        pad = torch.rand(T, generator=gen, device=DEVICE) < 0.09
        pad[0] = False
        ids = torch.where(pad[:, None], E, ids)
    flat = ids.flatten()
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    order = torch.sort(flat, stable=True).indices
    row = torch.empty_like(flat)
    row[order] = torch.arange(flat.numel(), device=DEVICE)
    row = torch.where(flat < E, row, -1)
    return counts.int(), (counts.cumsum(0) - counts).int(), row.int().view(T, k)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEVICE)  # noqa: E731
    empty = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=DEVICE)  # noqa: E731
    st = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_grad"):
        T, H = case["T"], case["H"]
        # a residual stream: some channels are far larger than the others
        loud = 1.0 + 20.0 * (torch.rand(H, generator=gen, device=DEVICE) < 0.01)
        st["weight"] = 1.0 + 0.2 * normal(H)
        if op == "norm":
            st["x"] = (normal(T, H) * loud).bfloat16()
            st["residual"] = normal(T, H).bfloat16() if case["residual"] else None
            st["total"] = empty(T, H) if case["residual"] else None
            st["y"] = empty(T, H) if case["y"] else None
            st["codes"] = empty(T, H, dtype=torch.uint8) if case["codes"] else None
            st["scales"] = empty(T, H // 128, dtype=torch.float32) if case["codes"] else None
            st["inv_rms"] = empty(T, dtype=torch.float32) if case["save"] else None
        else:
            st["total"] = (normal(T, H) * loud).bfloat16()
            t = st["total"].double()
            st["inv_rms"] = ((t * t).mean(1) + EPS).rsqrt().float()
            st["grad_y"] = (1e-2 * normal(T, H)).bfloat16()
            st["carried"] = (1e-2 * normal(T, H)).bfloat16() if case["carried"] else None
            st["grad_x"] = empty(T, H)
            st["grad_weight"] = empty(H, dtype=torch.float32)
        return st
    if op == "weights":
        E, P, K = case["E"], case["P"], case["K"]
        t = torch.bfloat16 if case["type"] == "bf16" else torch.float32
        st["w"] = torch.randn(E, P, K, generator=gen, device=DEVICE, dtype=t) * K ** -0.5
        st["codes"] = empty(E, P, K, dtype=torch.uint8)
        st["scales"] = empty(E, P // 128, K // 128, dtype=torch.float32)
        return st
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    R = T * k
    st["counts"], st["offsets"], st["token_row"] = _route(case, gen)
    st["longest"] = int(st["counts"].max())  # only the plain form's padded product needs it
    st["x"], st["x_scales"] = _blocks(normal(R, H), 1, 128)
    st["up"], st["up_scales"] = _blocks(normal(E, 2 * I, H) * H ** -0.5, 128, 128)
    st["down"], st["down_scales"] = _blocks(normal(E, H, I) * I ** -0.5, 128, 128)
    if op == "ffn":
        st["residual"] = normal(R, H).bfloat16() if case["residual"] else None
        st["y"] = empty(R, H)
        st["pre"] = empty(R, 2 * I) if case["save"] else None
    else:
        st["grad_y"] = (1e-2 * normal(R, H)).bfloat16()
        st["pre"] = normal(R, 2 * I).bfloat16()
        st["grad_x"] = empty(R, H)
        st["grad_up"] = empty(E, 2 * I, H)
        st["grad_down"] = empty(E, H, I)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_norm(st):
    case = st["case"]
    t = st["x"].float()
    out = {}
    if case["residual"]:
        out["total"] = (t + st["residual"].float()).bfloat16()
        t = out["total"].float()
    inv = 1.0 / torch.sqrt((t * t).mean(1, keepdim=True) + EPS)
    v = t * inv * st["weight"]
    if case["y"]:
        out["y"] = v.bfloat16()
    if case["codes"]:
        out["codes"], out["scales"] = _blocks(v, 1, 128)
    if case["save"]:
        out["inv_rms"] = inv.flatten()
    return out


def _plain_norm_grad(st):
    t, inv = st["total"].float(), st["inv_rms"][:, None]
    g = st["grad_y"].float()
    h = t * inv
    a = g * st["weight"]
    gx = inv * (a - h * (a * h).mean(1, keepdim=True))
    if st["carried"] is not None:
        gx = gx + st["carried"].float()
    return {"grad_x": gx.bfloat16(), "grad_weight": (g * h).sum(0)}


def _plain_weights(st):
    codes, scales = _blocks(st["w"].float(), 128, 128)
    return {"codes": codes, "scales": scales}


def _places(st):
    """Where each receive row sits in the padded [E, longest] form (rows of no
    segment at the end), and whether it is in a segment."""
    R, E = st["x"].shape[0], st["counts"].numel()
    r = torch.arange(R, device=DEVICE)
    e = torch.searchsorted((st["offsets"] + st["counts"]).long(), r, right=True)
    there = e < E
    e = e.clamp(max=E - 1)
    at = e * st["longest"] + r - st["offsets"][e]
    return torch.where(there, at, E * st["longest"]), there


def _pad(st, rows, at):
    E, M = st["counts"].numel(), st["longest"]
    full = torch.zeros(E * M + 1, rows.shape[1], device=DEVICE)
    full.index_copy_(0, at, rows)
    return full[:E * M].view(E, M, rows.shape[1])


def _unpad(padded, at, there):
    rows = padded.reshape(-1, padded.shape[-1])
    return torch.where(there[:, None], rows[at.clamp(max=rows.shape[0] - 1)], 0.0)


def _widen(codes, scales, rows):
    """fp32 values of e4m3 codes with one scale per rows x 128 block."""
    return codes.float() * scales.repeat_interleave(128, -1).repeat_interleave(rows, -2)


def _rounded(v):
    """fp32 values after the rounding to 8 bits in blocks of 128 columns."""
    return _widen(*_blocks(v, 1, 128), 1)


def _plain_ffn(st):
    I = st["case"]["I"]
    at, there = _places(st)
    x = _pad(st, _widen(st["x"], st["x_scales"], 1), at)
    z = torch.matmul(x, _widen(st["up"], st["up_scales"], 128).transpose(1, 2))
    g, u = z[..., :I], z[..., I:]
    h = _rounded((g / (1.0 + torch.exp(-g)) * u).reshape(-1, I)).view(g.shape)
    y = torch.matmul(h, _widen(st["down"], st["down_scales"], 128).transpose(1, 2))
    y = _unpad(y, at, there)
    if st["residual"] is not None:
        y = torch.where(there[:, None], y + st["residual"].float(), 0.0)
    out = {"y": y.bfloat16()}
    if st["pre"] is not None:
        out["pre"] = _unpad(z, at, there).bfloat16()
    return out


def _plain_ffn_grad(st):
    I = st["case"]["I"]
    at, there = _places(st)
    gy = torch.where(there[:, None], st["grad_y"].float(), 0.0)
    pre = torch.where(there[:, None], st["pre"].float(), 0.0)
    gh = torch.matmul(_pad(st, _rounded(gy), at), _widen(st["down"], st["down_scales"], 128))
    gh = _unpad(gh, at, there)
    g, u = pre[:, :I], pre[:, I:]
    s = 1.0 / (1.0 + torch.exp(-g))
    gz = torch.cat([gh * u * s * (1.0 + g * (1.0 - s)), gh * g * s], 1)
    gx = torch.matmul(_pad(st, _rounded(gz), at), _widen(st["up"], st["up_scales"], 128))
    x = torch.where(there[:, None], _widen(st["x"], st["x_scales"], 1), 0.0)
    gup = torch.matmul(_pad(st, gz, at).transpose(1, 2), _pad(st, x, at))
    gdown = torch.matmul(_pad(st, gy, at).transpose(1, 2), _pad(st, g * s * u, at))
    return {"grad_x": _unpad(gx, at, there).bfloat16(), "grad_up": gup.bfloat16(),
            "grad_down": gdown.bfloat16()}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(st):
    from combine_moe_dispatch_amd import api
    case = st["case"]
    op = case["op"]
    if op == "norm":
        api.moe_rms_norm(st["x"], st["residual"], st["weight"], EPS, st["total"], st["y"],
                         st["codes"], st["scales"], st["inv_rms"])
        out = {n: st[n] for n in ("total", "y", "scales", "inv_rms") if st[n] is not None}
        if case["codes"]:
            out["codes"] = st["codes"].view(E4M3)
        return out
    if op == "norm_grad":
        if "workspace" not in st:
            st["workspace"] = api.alloc_rms_norm_workspace(case["T"], case["H"], DEVICE)
        api.moe_rms_norm_backward(st["grad_y"], st["total"], st["weight"], st["inv_rms"],
                                  st["carried"], st["grad_x"], st["grad_weight"],
                                  st["workspace"])
        return {"grad_x": st["grad_x"], "grad_weight": st["grad_weight"]}
    if op == "weights":
        api.moe_quantize_weight(st["w"], st["codes"], st["scales"])
        return {"codes": st["codes"].view(E4M3), "scales": st["scales"]}
    none = st["counts"][:0]  # what these calls do not read
    lay = api.Layout(st["counts"], st["offsets"], none, none, st["token_row"], None, none)
    shape = api.Shape(case["T"], case["H"], case["E"], case["k"], 1, 0,
                      api.MOE_PAYLOAD_FP8_E4M3_B128)
    ffn = api.Ffn(case["H"], case["I"])
    weights = (st["up"], st["up_scales"], st["down"], st["down_scales"])
    if op == "ffn":
        if "workspace" not in st:
            st["workspace"] = api.alloc_ffn_workspace(shape, ffn, DEVICE)
        api.moe_expert_ffn(shape, ffn, st["x"], st["x_scales"], lay, *weights, st["residual"],
                           st["y"], st["pre"], st["workspace"])
        return {n: st[n] for n in ("y", "pre") if st[n] is not None}
    if "workspace" not in st:
        st["workspace"] = api.alloc_ffn_workspace(shape, ffn, DEVICE, backward=True)
    api.moe_expert_ffn_backward(shape, ffn, st["grad_y"], st["x"], st["x_scales"], lay, *weights,
                                st["pre"], st["grad_x"], st["grad_up"], st["grad_down"],
                                st["workspace"])
    return {n: st[n] for n in ("grad_x", "grad_up", "grad_down")}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "weights": _plain_weights,
          "ffn": _plain_ffn, "ffn_grad": _plain_ffn_grad}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        row = 2 * H * (1 + 2 * case["residual"] + case["y"]) + 4 * case["save"]
        row += (H + H // 32) * case["codes"]
        return {"bytes": T * row + 4 * H, "flops": 4 * T * H}
    if op == "norm_grad":
        T, H = case["T"], case["H"]
        return {"bytes": T * (2 * H * (3 + case["carried"]) + 4) + 8 * H, "flops": 9 * T * H}
    if op == "weights":
        n = case["E"] * case["P"] * case["K"]
        return {"bytes": n * (5 if case["type"] == "fp32" else 3) + n // 4096, "flops": 2 * n}
    E, H, I = case["E"], case["H"], case["I"]
    R = case["T"] * case["k"]
    weights = min(E, R) * 3 * H * I  # of the experts that have rows
    if op == "ffn":
        row = H + H // 32 + 2 * H * (1 + case["residual"]) + 4 * I * case["save"]
        return {"bytes": weights + weights // 4096 + R * row, "flops": 6 * R * H * I}
    row = 2 * H + H + H // 32 + 4 * I + 2 * H
    return {"bytes": weights + weights // 4096 + 6 * E * H * I + R * row, "flops": 12 * R * H * I}


# ---------------------------------------------------------------------------
# the definitions in fp64
# ---------------------------------------------------------------------------
def _exact_e4m3(v):
    """The nearest e4m3 values (fp64, ties to even), magnitudes cut at 448."""
    exponent = torch.frexp(v).exponent - 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_codes(v):
    """e4m3 values and scales of the rows of v in blocks of 128 columns.  Scale
    and quotient are fp32 numbers by definition: 16-bit values often lie on the
    border between two codes, where any other quotient is another code."""
    parts = v.unflatten(-1, (-1, 128))
    scale = (parts.abs().amax(-1) / 448.0).float()
    quotient = torch.where(scale[..., None] > 0, parts.float() / scale[..., None], 0.0)
    return _exact_e4m3(quotient.double()).flatten(-2), scale.double()


def _exact_values(v):
    codes, scale = _exact_codes(v)
    return (codes.unflatten(-1, (-1, 128)) * scale[..., None]).flatten(-2)


def _exact_block(codes, scales):
    """Values of one expert's weight: codes times their 128 x 128 block's scale."""
    P, K = codes.shape
    w = codes.double().view(P // 128, 128, K // 128, 128)
    return (w * scales.double()[:, None, :, None]).reshape(P, K)


def _exact_norm(st):
    case = st["case"]
    out = {}
    t = st["x"].double()
    if case["residual"]:
        out["total"] = t + st["residual"].double()
        t = out["total"].bfloat16().double()  # what the next layer is given
    w = st["weight"].double()
    inv = (t.square().mean(1) + EPS).rsqrt()
    v = t * inv[:, None] * w
    if case["y"]:
        out["y"] = v
    if case["codes"]:
        out["codes"], out["scales"] = _exact_codes(v)
    if case["save"]:
        out["inv_rms"] = inv
    return out


def _exact_norm_grad(st):
    t = st["total"].double()
    w = st["weight"].double()
    g, inv = st["grad_y"].double(), st["inv_rms"].double()[:, None]
    # d y_j / d t_i = w_j inv (1[i = j] - t_i t_j inv^2 / H)
    gw = g * w
    gx = gw * inv - t * ((gw * t).sum(1, keepdim=True) * inv ** 3 / t.shape[1])
    if st["carried"] is not None:
        gx = gx + st["carried"].double()
    return {"grad_x": gx, "grad_weight": torch.einsum("th,th->h", g, t * inv)}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(st)
    if op == "norm_grad":
        return _exact_norm_grad(st)
    if op == "weights":
        E, P, K = st["w"].shape
        codes = torch.empty(E, P, K, dtype=torch.float32, device=DEVICE)  # e4m3 values: exact
        scales = torch.empty(E, P // 128, K // 128, dtype=torch.float64, device=DEVICE)
        for e in range(E):
            # fp32 scales and quotients, as in _exact_codes
            b = st["w"][e].view(P // 128, 128, K // 128, 128)
            s = (b.double().abs().amax(dim=(1, 3)) / 448.0).float()
            codes[e] = _exact_e4m3((b.float() / s[:, None, :, None]).double()).view(P, K).float()
            scales[e] = s.double()
        return {"codes": codes, "scales": scales}
    H, I = case["H"], case["I"]
    E, R = case["E"], st["x"].shape[0]
    silu = torch.nn.functional.silu
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64, device=DEVICE)  # noqa: E731
    if op == "ffn":
        out = {"y": zeros(R, H)}
        if case["save"]:
            out["pre"] = zeros(R, 2 * I)
    else:
        out = {"grad_x": zeros(R, H), "grad_up": zeros(E, 2 * I, H), "grad_down": zeros(E, H, I)}
    for e, (a, n) in enumerate(zip(st["offsets"].tolist(), st["counts"].tolist())):
        if n == 0:
            continue
        s = slice(a, a + n)
        x = (st["x"][s].double().unflatten(1, (-1, 128)) *
             st["x_scales"][s].double()[..., None]).flatten(1)
        up = _exact_block(st["up"][e], st["up_scales"][e])
        down = _exact_block(st["down"][e], st["down_scales"][e])
        if op == "ffn":
            z = x @ up.T
            gate, value = z.chunk(2, 1)
            y = _exact_values(silu(gate) * value) @ down.T
            if st["residual"] is not None:
                y = y + st["residual"][s].double()
            out["y"][s] = y
            if case["save"]:
                out["pre"][s] = z
            continue
        gy = st["grad_y"][s].double()
        z = st["pre"][s].double().requires_grad_()
        gate, value = z.chunk(2, 1)
        h = silu(gate) * value
        gz, = torch.autograd.grad(h, z, _exact_values(gy) @ down)
        out["grad_x"][s] = _exact_values(gz) @ up
        out["grad_up"][e] = gz.T @ x
        out["grad_down"][e] = gy.T @ h.detach()
    return out
