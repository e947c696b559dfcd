"""The operators around dispatch and combine, as cases that can be timed.

Operators: the router's balance loss with its per-expert counts; the router's
gradient (of the routed weights and of the balance loss); the combine's
gradient; the experts' matrix product with bias, activation and residual; and
that product's gradient.

`run` computes a case in its plain form, elementary torch operations in fp32
rounded once at the end, or with `own` set through this library's calls.
`exact` gives the same results in fp64, from the definitions.

Receive rows are packed: expert segments back to back in expert order, inside
a segment the (token, slot) pairs ascending.  A padded token has no expert
(all its ids are -1) and its pairs have no row.
"""
import math

import torch

own = False

DEVICE = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a 16-token step of the smallest configured layer: pure call latency
        {"name": "balance_tiny", "op": "balance", "T": 16, "E": 8, "k": 2, "score": "softmax",
         "bias": False, "seqs": 0, "padded": False},
        # one prefill-sized micro-batch of ragged sequences with padded tokens
        {"name": "balance_prefill", "op": "balance", "T": 4096, "E": 256, "k": 8,
         "score": "sigmoid", "bias": True, "seqs": 5, "padded": True},
        # the router's gradient for a decode-sized batch, 384 experts
        {"name": "route_grad_small", "op": "route_grad", "T": 128, "E": 384, "k": 8,
         "score": "sigmoid", "bias": True, "seqs": 0, "padded": False},
        # a long training batch of many ragged sequences
        {"name": "route_grad_long", "op": "route_grad", "T": 65536, "E": 256, "k": 8,
         "score": "softmax", "bias": True, "seqs": 37, "padded": True},
        # the combine's gradient at the decode shape
        {"name": "combine_grad_small", "op": "combine_grad", "T": 128, "H": 7168, "E": 256,
         "k": 8, "padded": False},
        # and at the prefill shape
        {"name": "combine_grad_prefill", "op": "combine_grad", "T": 4096, "H": 7168, "E": 256,
         "k": 8, "padded": True},
        # one token at the gate/up projection: the chosen experts' weights are streamed
        {"name": "matmul_token", "op": "matmul", "T": 1, "E": 32, "k": 8, "K": 7168, "F": 2048,
         "act": "swiglu", "type": "bf16", "bias": False, "residual": False, "save": False,
         "padded": False},
        # fp8 serving: block-scaled tokens times block-scaled weights
        {"name": "matmul_fp8", "op": "matmul", "T": 512, "E": 32, "k": 8, "K": 7168, "F": 2048,
         "act": "swiglu", "type": "fp8", "bias": False, "residual": False, "save": False,
         "padded": False},
        # the shared expert's down projection added to the routed sum, odd token count
        {"name": "matmul_shared", "op": "matmul", "T": 1021, "E": 1, "k": 1, "K": 2048, "F": 7168,
         "act": "none", "type": "bf16", "bias": True, "residual": True, "save": False,
         "padded": False},
        # gate/up projection of a prefill, pre-activations kept for the backward pass
        {"name": "matmul_prefill", "op": "matmul", "T": 4096, "E": 32, "k": 8, "K": 7168,
         "F": 2048, "act": "swiglu", "type": "bf16", "bias": True, "residual": False,
         "save": True, "padded": True},
        # gradients of a small layer of odd sizes
        {"name": "matmul_grad_odd", "op": "matmul_grad", "T": 301, "E": 6, "k": 2, "K": 1432,
         "F": 712, "act": "silu", "padded": True},
        # gradients of the gate/up projection
        {"name": "matmul_grad", "op": "matmul_grad", "T": 1024, "E": 32, "k": 8, "K": 7168,
         "F": 2048, "act": "swiglu", "padded": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "route_grad", "combine_grad", "matmul", "matmul", "matmul",
                     "matmul_grad"])
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("balance", "route_grad"):
        E = rng.randint(2, 384)
        return {"op": op, "T": _log_int(rng, 1, 32768), "E": E, "k": rng.randint(1, min(E, 12)),
                "score": rng.choice(["sigmoid", "softmax"]), "bias": yes(),
                "seqs": rng.choice([0, 1, rng.randint(2, 64)]), "padded": yes()}
    if op == "combine_grad":
        E = rng.randint(8, 256)
        return {"op": op, "T": _log_int(rng, 1, 3000), "H": 8 * _log_int(rng, 16, 896), "E": E,
                "k": rng.randint(1, 8), "padded": yes()}
    E = rng.choice([1, rng.randint(2, 32), rng.randint(8, 32)])
    k = rng.randint(1, min(E, 8))
    act = rng.choice(["none", "silu", "gelu", "swiglu", "swiglu"])
    if op == "matmul" and yes():
        K, F = 128 * _log_int(rng, 1, 56), 128 * _log_int(rng, 1, 28)
        return {"op": op, "T": _log_int(rng, 1, 4096), "E": E, "k": k, "K": K, "F": F, "act": act,
                "type": "fp8", "bias": yes(), "residual": yes(), "save": False, "padded": yes()}
    K, F = 8 * _log_int(rng, 12, 896), 8 * _log_int(rng, 12, 256)
    if op == "matmul":
        return {"op": op, "T": _log_int(rng, 1, 4096), "E": E, "k": k, "K": K, "F": F, "act": act,
                "type": "bf16", "bias": yes(), "residual": yes(), "save": yes(), "padded": yes()}
    return {"op": op, "T": _log_int(rng, 1, 1024), "E": E, "k": k, "K": K, "F": F, "act": act,
            "padded": yes()}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _padded(case, gen):
    """Which tokens are padding: none, or about one in eleven (never all)."""
    T = case["T"]
    if not case["padded"]:
        return torch.zeros(T, dtype=torch.bool, device=DEVICE)
    pad = torch.rand(T, generator=gen, device=DEVICE) < 0.09
    pad[0] = False
    return pad


def _pairs(ids, E):
    """Packed layout of an id list: counts, offsets, row of each pair (-1: none)."""
    flat = ids.flatten().long()
    bucket = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = torch.bincount(bucket, minlength=E + 1)[:E]
    order = torch.sort(bucket, stable=True).indices
    row = torch.empty_like(flat)
    row[order] = torch.arange(flat.numel(), device=DEVICE)
    row = torch.where(bucket < E, row, -1)
    offsets = counts.cumsum(0) - counts
    return counts.int(), offsets.int(), row.int().view(ids.shape)


def _fp8_blocks(t, rows, cols):
    """e4m3 codes and fp32 scales of a [..., R, C] tensor in blocks of rows x cols."""
    R, C = t.shape[-2], t.shape[-1]
    b = t.view(*t.shape[:-2], R // rows, rows, C // cols, cols)
    scale = b.abs().amax(dim=(-3, -1)) / 448.0
    codes = b / scale[..., :, None, :, None]
    return codes.reshape(t.shape).to(torch.float8_e4m3fn), scale.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEVICE)  # noqa: E731
    T, k, E = case["T"], case["k"], case["E"]
    st = {"case": case}
    pad = _padded(case, gen)
    logits = normal(T, E)
    if case["op"] in ("balance", "route_grad"):
        st["logits"] = logits
        st["bias"] = 0.5 * normal(E) if case["bias"] else None
        biased = logits if st["bias"] is None else logits + st["bias"]
        top = torch.topk(biased, k, dim=1)
        s = torch.sigmoid(top.values) if case["score"] == "sigmoid" else \
            torch.exp(top.values - top.values[:, :1])
        st["weights"] = s / s.sum(1, keepdim=True)
        st["ids"] = torch.where(pad[:, None], -1, top.indices).int()
        st["offsets"] = None
        S = 1
        if case["seqs"]:
            S = case["seqs"]
            cuts = torch.randint(0, T + 1, (S + 1,), generator=gen, device=DEVICE).sort().values
            cuts[0] = 0
            st["offsets"] = cuts.int()
        st["coef"] = 1e-2
        if case["op"] == "route_grad":
            # what the forward pass left: counts per sequence, tokens per sequence
            seq, valid = _sequences(st)
            at = torch.where((st["ids"] >= 0) & valid[:, None], seq[:, None] * E + st["ids"], S * E)
            st["counts"] = torch.bincount(at.flatten(), minlength=S * E + 1)[:S * E].int().view(S, E)
            st["tokens"] = torch.bincount(torch.where(valid, seq, S), minlength=S + 1)[:S].int()
            st["grad_weights"] = torch.where(pad[:, None], 0.0, 0.02 * normal(T, k))
            st["grad_loss"] = torch.ones(1, device=DEVICE)
        return st
    ids = torch.topk(logits, k, dim=1).indices
    ids = torch.where(pad[:, None], -1, ids).int()
    st["counts"], st["row_offsets"], st["token_row"] = _pairs(ids, E)
    st["ids"] = ids
    R = T * k
    if case["op"] == "combine_grad":
        H = case["H"]
        st["grad_out"] = normal(T, H).bfloat16()
        st["y"] = normal(R, H).bfloat16()
        w = torch.rand(T, k, generator=gen, device=DEVICE) + 0.05
        st["weights"] = w / w.sum(1, keepdim=True)
        st["grad_y"] = torch.zeros(R, H, dtype=torch.bfloat16, device=DEVICE)
        return st
    K, F = case["K"], case["F"]
    P = 2 * F if case["act"] == "swiglu" else F
    st["longest"] = int(st["counts"].max())  # only the plain form's padded product needs it
    w = torch.randn(E, P, K, generator=gen, device=DEVICE,
                    dtype=torch.float32 if case.get("type") == "fp8" else torch.bfloat16)
    w *= K ** -0.5
    x = normal(R, K)
    if case.get("type") == "fp8":
        st["w"], st["w_scales"] = _fp8_blocks(w, 128, 128)
        st["x"], st["x_scales"] = _fp8_blocks(x, 1, 128)
    else:
        st["w"], st["x"] = w, x.bfloat16()
    if case["op"] == "matmul":
        st["bias"] = 0.3 * normal(E, P) if case["bias"] else None
        st["residual"] = normal(R, F).bfloat16() if case["residual"] else None
        st["y"] = torch.zeros(R, F, dtype=torch.bfloat16, device=DEVICE)
        st["pre"] = torch.zeros(R, P, dtype=torch.bfloat16, device=DEVICE) if case["save"] else None
        return st
    st["grad_y"] = normal(R, F).bfloat16()
    st["pre"] = normal(R, P).bfloat16()
    st["grad_x"] = torch.zeros(R, K, dtype=torch.bfloat16, device=DEVICE)
    st["grad_w"] = torch.empty_like(w)
    st["grad_b"] = torch.empty(E, P, device=DEVICE)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _sequences(st):
    """Each token's sequence, and whether it counts: inside a sequence and with
    an expert to go to."""
    ids, off = st["ids"], st["offsets"]
    T, E = st["logits"].shape
    some = ((ids >= 0) & (ids < E)).any(1)
    if off is None:
        return torch.zeros(T, dtype=torch.long, device=DEVICE), some
    t = torch.arange(T, device=DEVICE, dtype=torch.int32)
    seq = torch.searchsorted(off, t, right=True) - 1
    return seq, some & (seq >= 0) & (seq < off.numel() - 1)


def _scores(st):
    """Probabilities p [T, E] (each row sums to one) and, for sigmoid scores, s."""
    l = st["logits"] if st["bias"] is None else st["logits"] + st["bias"]
    if st["case"]["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
        return s / s.sum(1, keepdim=True), s
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True), None


def _plain_balance(st):
    T, E = st["logits"].shape
    S = 1 if st["offsets"] is None else st["offsets"].numel() - 1
    k, ids = st["ids"].shape[1], st["ids"]
    seq, valid = _sequences(st)
    p, _ = _scores(st)
    member = ((seq[None, :] == torch.arange(S, device=DEVICE)[:, None]) & valid).float()
    n = member.sum(1)
    at = torch.where((ids >= 0) & (ids < E) & valid[:, None], seq[:, None] * E + ids, S * E)
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device=DEVICE)
    counts.index_add_(0, at.flatten(), torch.ones(T * k, dtype=torch.int32, device=DEVICE))
    counts = counts[:S * E].view(S, E)
    m = n.clamp(min=1.0)[:, None]
    probs = (member @ p) / m
    loss = (st["coef"] / S) * (counts.float() * (E / k) / m * probs).sum()
    return {"counts": counts, "tokens": n.int(), "probs": probs, "loss": loss.view(1)}


def _plain_route_grad(st):
    T, E = st["logits"].shape
    S, k, ids = st["counts"].shape[0], st["ids"].shape[1], st["ids"]
    seq, valid = _sequences(st)
    p, s = _scores(st)
    n = st["tokens"].float().clamp(min=1.0)[:, None]
    g = (st["coef"] / S) * st["grad_loss"] * (E / k) * st["counts"].float() / (n * n)
    g = torch.where(valid[:, None], g[seq.clamp(0, S - 1)], 0.0)
    grad = p * (g - (g * p).sum(1, keepdim=True))
    there = (ids >= 0) & (ids < E)
    at = torch.where(there, ids, 0).long()
    gw = torch.where(there, st["grad_weights"], 0.0)
    w = st["weights"]
    gl = torch.where(there, w * (gw - (gw * w).sum(1, keepdim=True)), 0.0)
    if s is not None:
        grad = grad * (1.0 - s)
        gl = gl * (1.0 - s.gather(1, at))
    grad.scatter_add_(1, at, gl)
    return {"logits": grad, "bias": None if st["bias"] is None else grad.sum(0)}


def _plain_combine_grad(st):
    T, k = st["token_row"].shape
    R, H = st["y"].shape
    row = st["token_row"].flatten().long()
    there = (row >= 0)[:, None]
    go = st["grad_out"].float().repeat_interleave(k, 0)
    y = st["y"].float()[row.clamp(min=0)]
    gw = torch.where(there, (go * y).sum(1, keepdim=True), 0.0)
    gy = torch.zeros(R + 1, H, device=DEVICE)  # the pairs without a row share the last one
    gy.index_copy_(0, torch.where(row >= 0, row, R), st["weights"].view(-1, 1) * go)
    return {"grad_y": gy[:R].bfloat16(), "grad_weights": gw.view(T, k)}


def _places(st):
    """Where each receive row sits in the padded [E, longest] form (rows of no
    segment at the end), and whether it is in a segment."""
    R, E = st["x"].shape[0], st["counts"].numel()
    r = torch.arange(R, device=DEVICE)
    ends = (st["row_offsets"] + st["counts"]).long()
    e = torch.searchsorted(ends, r, right=True)
    there = e < E
    e = e.clamp(max=E - 1)
    at = e * st["longest"] + r - st["row_offsets"][e]
    return torch.where(there, at, E * st["longest"]), there, e


def _pad(st, rows, at):
    E, M = st["counts"].numel(), st["longest"]
    full = torch.zeros(E * M + 1, rows.shape[1], device=DEVICE)
    full.index_copy_(0, at, rows)
    return full[:E * M].view(E, M, rows.shape[1])


def _widen(codes, scales, rows):
    """fp32 values of e4m3 codes with one scale per rows x 128 block."""
    return codes.float() * scales.repeat_interleave(128, -1).repeat_interleave(rows, -2)


def _act(name, z):
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "swiglu":
        F = z.shape[-1] // 2
        g, u = z[..., :F], z[..., F:]
        return g / (1.0 + torch.exp(-g)) * u
    return z


def _act_grad(name, z, gy):
    """Gradient of sum(gy * act(z)) with respect to z."""
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return gy * s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return gy * (cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    if name == "swiglu":
        F = z.shape[-1] // 2
        g, u = z[..., :F], z[..., F:]
        s = 1.0 / (1.0 + torch.exp(-g))
        return torch.cat([gy * u * s * (1.0 + g * (1.0 - s)), gy * g * s], -1)
    return gy


def _plain_matmul(st):
    case = st["case"]
    E = case["E"]
    at, there, e = _places(st)
    if case["type"] == "fp8":
        x, w = _widen(st["x"], st["x_scales"], 1), _widen(st["w"], st["w_scales"], 128)
    else:
        x, w = st["x"].float(), st["w"].float()
    z = torch.matmul(_pad(st, x, at), w.transpose(1, 2)).view(E * st["longest"], -1)
    z = torch.where(there[:, None], z[at.clamp(max=E * st["longest"] - 1)], 0.0)
    if st["bias"] is not None:
        z = z + st["bias"][e]
    y = _act(case["act"], z)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    out = {"y": torch.where(there[:, None], y, 0.0).bfloat16()}
    if case["save"]:
        out["pre"] = torch.where(there[:, None], z, 0.0).bfloat16()
    return out


def _plain_matmul_grad(st):
    case = st["case"]
    E = case["E"]
    at, there, _ = _places(st)
    gz = _act_grad(case["act"], st["pre"].float(), st["grad_y"].float())
    gz = _pad(st, torch.where(there[:, None], gz, 0.0), at)
    gx = torch.matmul(gz, st["w"].float()).view(E * st["longest"], -1)
    gx = torch.where(there[:, None], gx[at.clamp(max=E * st["longest"] - 1)], 0.0)
    gw = torch.matmul(gz.transpose(1, 2), _pad(st, st["x"].float(), at))
    return {"grad_x": gx.bfloat16(), "grad_w": gw.bfloat16(), "grad_b": gz.sum(1)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _layout(api, st):
    none = st["counts"][:0]  # what these calls do not read
    return api.Layout(st["counts"], st["row_offsets"], none, none, st["token_row"], None, none)


def _own(st):
    from combine_moe_dispatch_amd import api
    case = st["case"]
    if case["op"] in ("balance", "route_grad"):
        score = api.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else api.MOE_SCORE_SOFTMAX
    if case["op"] == "balance":
        loss, counts, probs, tokens = api.moe_balance_loss(
            st["logits"], st["bias"], st["ids"], score, st["coef"], st["offsets"])
        return {"counts": counts, "tokens": tokens, "probs": probs, "loss": loss}
    if case["op"] == "route_grad":
        logits, bias = api.moe_route_backward(
            st["logits"], st["bias"], st["ids"], st["weights"], st["grad_weights"], score,
            coef=st["coef"], seq_offsets=st["offsets"], expert_counts=st["counts"],
            seq_tokens=st["tokens"], grad_loss=st["grad_loss"], with_grad_bias=case["bias"])
        return {"logits": logits, "bias": bias}
    lay = _layout(api, st)
    if case["op"] == "combine_grad":
        shape = api.Shape(case["T"], case["H"], case["E"], case["k"], 1, 0)
        grad_weights = torch.empty_like(st["weights"])
        api.moe_combine_backward(shape, st["grad_out"], st["y"], lay, st["weights"],
                                 st["grad_y"], grad_weights)
        return {"grad_y": st["grad_y"], "grad_weights": grad_weights}
    act = {"none": api.MOE_ACT_NONE, "silu": api.MOE_ACT_SILU, "gelu": api.MOE_ACT_GELU,
           "swiglu": api.MOE_ACT_SWIGLU}[case["act"]]
    lin = api.Linear(case["K"], case["F"], act)
    fp8 = case.get("type") == "fp8"
    shape = api.Shape(case["T"], case["K"], case["E"], case["k"], 1, 0,
                      api.MOE_PAYLOAD_FP8_E4M3_B128 if fp8 else api.MOE_PAYLOAD_BF16)
    if case["op"] == "matmul":
        api.moe_expert_matmul(shape, lin, st["x"], st["x_scales"] if fp8 else None, lay, st["w"],
                              st["w_scales"] if fp8 else None, st["bias"], st["residual"],
                              st["y"], st["pre"])
        return {"y": st["y"], "pre": st["pre"]} if case["save"] else {"y": st["y"]}
    if "workspace" not in st:
        st["workspace"] = api.alloc_expert_workspace(shape, lin, DEVICE)
    api.moe_expert_matmul_backward(shape, lin, st["grad_y"], st["x"], lay, st["w"], st["pre"],
                                   st["grad_x"], st["grad_w"], st["grad_b"], st["workspace"])
    return {"grad_x": st["grad_x"], "grad_w": st["grad_w"], "grad_b": st["grad_b"]}


_PLAIN = {"balance": _plain_balance, "route_grad": _plain_route_grad,
          "combine_grad": _plain_combine_grad, "matmul": _plain_matmul,
          "matmul_grad": _plain_matmul_grad}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    S = max(1, case.get("seqs", 0))
    R = T * k
    if case["op"] == "balance":
        return {"bytes": 4 * T * E + 4 * R + 8 * S * E + 4 * E * case["bias"], "flops": 6 * T * E}
    if case["op"] == "route_grad":
        return {"bytes": 8 * T * E + 12 * R + 4 * S * E + 8 * E * case["bias"],
                "flops": 12 * T * E}
    if case["op"] == "combine_grad":
        H = case["H"]
        return {"bytes": 2 * T * H + 4 * R * H + 12 * R, "flops": 3 * R * H}
    K, F = case["K"], case["F"]
    P = 2 * F if case["act"] == "swiglu" else F
    one = 1 if case.get("type") == "fp8" else 2
    busy = min(E, R)  # experts whose weights are needed
    if case["op"] == "matmul":
        rows = R * (K * one + 2 * F * (1 + case["residual"]) + 2 * P * case["save"])
        return {"bytes": busy * P * K * one + rows + 4 * E * P * case["bias"],
                "flops": 2 * R * P * K}
    rows = 2 * R * (F + 2 * K + (P if case["act"] != "none" else 0))
    return {"bytes": 2 * busy * P * K + 2 * E * P * K + rows + 4 * E * P, "flops": 4 * R * P * K}


# ---------------------------------------------------------------------------
# the definitions in fp64
# ---------------------------------------------------------------------------
def _exact_balance_loss(l, score, ids, spans, coef):
    """Balance loss of biased logits l (fp64), with the means and the counts."""
    T, E = l.shape
    k = ids.shape[1]
    if score == "sigmoid":
        p = torch.sigmoid(l)
        p = p / p.sum(1, keepdim=True)
    else:
        p = torch.softmax(l, 1)
    loss = l.new_zeros(())
    means, counts, tokens = [], [], []
    for a, b in spans:
        keep = (ids[a:b] >= 0).any(1)
        n = int(keep.sum())
        part = ids[a:b][keep].flatten().long()
        c = torch.bincount(part[part >= 0], minlength=E).to(l)
        m = p[a:b][keep].sum(0) / max(n, 1)
        loss = loss + coef / len(spans) * (E * c / (k * max(n, 1)) * m).sum()
        means.append(m)
        counts.append(c)
        tokens.append(n)
    return loss, torch.stack(means), torch.stack(counts), tokens


def _exact_activation(name, z):
    if name == "silu":
        return torch.nn.functional.silu(z)
    if name == "gelu":
        return torch.nn.functional.gelu(z)
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        return torch.nn.functional.silu(g) * u
    return z


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("balance", "route_grad"):
        T = case["T"]
        cuts = [0, T] if st["offsets"] is None else st["offsets"].tolist()
        spans = list(zip(cuts[:-1], cuts[1:]))
        l = st["logits"].double().requires_grad_()
        b = None if st["bias"] is None else st["bias"].double().requires_grad_()
        biased = l if b is None else l + b
        loss, means, _, _ = _exact_balance_loss(biased, case["score"], st["ids"], spans, st["coef"])
        if case["op"] == "balance":
            return {"counts": None, "tokens": None, "probs": means.detach(),
                    "loss": loss.detach().view(1)}
        real = st["ids"] >= 0
        v = biased.gather(1, st["ids"].clamp(min=0).long())
        s = torch.sigmoid(v) if case["score"] == "sigmoid" else torch.softmax(v, 1)
        w = s / s.sum(1, keepdim=True)
        total = loss + (torch.where(real, st["grad_weights"].double(), 0.0) * w).sum()
        grads = torch.autograd.grad(total, [l] if b is None else [l, b])
        return {"logits": grads[0], "bias": None if b is None else grads[1]}
    if case["op"] == "combine_grad":
        row = st["token_row"]
        gy = torch.zeros(st["y"].shape, dtype=torch.float64, device=DEVICE)
        gw = torch.zeros(row.shape, dtype=torch.float64, device=DEVICE)
        go = st["grad_out"].double()
        for j in range(case["k"]):
            t = (row[:, j] >= 0).nonzero().flatten()
            r = row[t, j].long()
            gy[r] = st["weights"][t, j].double()[:, None] * go[t]
            gw[t, j] = (st["y"][r].double() * go[t]).sum(1)
        return {"grad_y": gy, "grad_weights": gw}
    P = st["w"].shape[1]
    ends = [(int(o), int(o) + int(c)) for o, c in
            zip(st["row_offsets"].tolist(), st["counts"].tolist())]
    R = st["x"].shape[0]
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64, device=DEVICE)  # noqa: E731
    if case["op"] == "matmul":
        y, pre = zeros(R, case["F"]), zeros(R, P)
        for e, (a, b) in enumerate(ends):
            if a == b:
                continue
            x, w = st["x"][a:b].double(), st["w"][e].double()
            if case["type"] == "fp8":
                x = (x.view(b - a, -1, 128) * st["x_scales"][a:b].double()[:, :, None]).view(b - a, -1)
                w = w.view(P // 128, 128, -1, 128) * st["w_scales"][e].double()[:, None, :, None]
                w = w.view(P, -1)
            z = x @ w.T
            if st["bias"] is not None:
                z = z + st["bias"][e].double()
            out = _exact_activation(case["act"], z)
            if st["residual"] is not None:
                out = out + st["residual"][a:b].double()
            y[a:b], pre[a:b] = out, z
        return {"y": y, "pre": pre} if case["save"] else {"y": y}
    gx, gw, gb = zeros(R, case["K"]), zeros(*st["w"].shape), zeros(case["E"], P)
    for e, (a, b) in enumerate(ends):
        if a == b:
            continue
        z = st["pre"][a:b].double().requires_grad_()
        out = _exact_activation(case["act"], z)
        gz = torch.autograd.grad((out * st["grad_y"][a:b].double()).sum(), z)[0]
        gx[a:b] = gz @ st["w"][e].double()
        gw[e] = gz.T @ st["x"][a:b].double()
        gb[e] = gz.sum(0)
    return {"grad_x": gx, "grad_w": gw, "grad_b": gb}
