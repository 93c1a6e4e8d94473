"""Cases of the feed-forward operators, and their plain forms.

Three operators of a serving step's feed-forward half:

* ``route``    scores of a token's experts, chosen by group and score, and
               their renormalised weights
* ``experts``  the chosen experts' MXFP4 products: up, gated activation,
               down, and the weighted sum over a token's experts
* ``linear``   the MXFP4 linear with bias, activation and residual in its
               epilogue, gated or not

``own`` chooses what :func:`run` does: the plain form in torch's elementary
operations, or the calls of :mod:`mxfp4_block_scaled_quant_amd`.
"""

import math
import random

import torch

own = False

DEVICE = "cuda"
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]     # magnitudes of the E2M1 codes


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token's choice among few experts: nothing but latency
        {"name": "route_one", "op": "route", "tokens": 1, "experts": 64, "top": 6, "groups": 1, "kept": 1,
         "scoring": "softmax", "bias": False, "type": "bfloat16", "padding": 0},
        # a decoding step's batch, three of its rows padding of a captured graph
        {"name": "route_step", "op": "route", "tokens": 61, "experts": 256, "top": 8, "groups": 8, "kept": 4,
         "scoring": "sigmoid", "bias": True, "type": "float32", "padding": 3},
        # a prompt's tokens
        {"name": "route_prompt", "op": "route", "tokens": 16001, "experts": 256, "top": 8, "groups": 8, "kept": 4,
         "scoring": "sigmoid", "bias": True, "type": "float32", "padding": 0},
        # one conversation: eight experts' weights streamed for one row each
        {"name": "experts_one", "op": "experts", "tokens": 1, "experts": 64, "top": 8, "hidden": 5120, "inner": 1024,
         "ranks": 1, "bias": False, "residual": True},
        # a decoding step of a full batch: every expert's weights, few rows each
        {"name": "experts_step", "op": "experts", "tokens": 61, "experts": 64, "top": 8, "hidden": 5120, "inner": 1024,
         "ranks": 1, "bias": False, "residual": True},
        # a chunk of prompts where this GPU holds a quarter of the experts
        {"name": "experts_chunk_shard", "op": "experts", "tokens": 1531, "experts": 32, "top": 6, "hidden": 5120,
         "inner": 1504, "ranks": 4, "bias": True, "residual": False},
        # whole prompts: the matrix units' side
        {"name": "experts_prompt", "op": "experts", "tokens": 8192, "experts": 64, "top": 8, "hidden": 5120,
         "inner": 1024, "ranks": 1, "bias": False, "residual": True},
        # one token through a feed-forward's gated half
        {"name": "linear_gate_one", "op": "linear", "tokens": 1, "rows": 34816, "hidden": 5120, "gated": True,
         "activation": "silu", "bias": False, "residual": False},
        # a decoding step's way back into the residual stream
        {"name": "linear_back_step", "op": "linear", "tokens": 37, "rows": 5120, "hidden": 14336, "gated": False,
         "activation": "none", "bias": True, "residual": True},
        # a chunk of a prompt through a plain feed-forward's first half
        {"name": "linear_gelu_chunk", "op": "linear", "tokens": 511, "rows": 14336, "hidden": 5120, "gated": False,
         "activation": "gelu_tanh", "bias": True, "residual": False},
        # a prompt through a feed-forward's gated half
        {"name": "linear_gate_prompt", "op": "linear", "tokens": 4096, "rows": 34816, "hidden": 5120, "gated": True,
         "activation": "silu", "bias": False, "residual": False},
        # a prompt's way back into the residual stream
        {"name": "linear_back_prompt", "op": "linear", "tokens": 8192, "rows": 5120, "hidden": 14336, "gated": False,
         "activation": "none", "bias": True, "residual": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "linear", "linear"])
    if op == "route":
        experts, groups, kept = rng.choice([(8, 1, 1), (60, 1, 1), (64, 1, 1), (64, 8, 3), (128, 1, 1), (160, 8, 3),
                                            (256, 8, 4), (256, 1, 1), (384, 1, 1), (512, 16, 6)])
        return {"op": op, "tokens": _log(rng, 1, 16000), "experts": experts, "top": rng.choice([1, 2, 4, 6, 8]),
                "groups": groups, "kept": kept, "scoring": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.choice([True, False]), "type": rng.choice(["float32", "bfloat16"]),
                "padding": rng.choice([0, 0, 2, 5])}
    if op == "experts":
        experts, top = rng.choice([(8, 2), (16, 4), (32, 4), (32, 8), (64, 6), (64, 8), (128, 8)])
        hidden = 32 * _log(rng, 32, 160)
        inner = 32 * _log(rng, 8, 1500000 // hidden // experts)
        tokens = _log(rng, 1, 6000)
        ranks = rng.choice([1, 1, 2, 4]) if tokens * top >= 64 else 1     # some pair meets an expert of this GPU
        return {"op": op, "tokens": tokens, "experts": experts, "top": top, "hidden": hidden,
                "inner": inner, "ranks": ranks, "bias": rng.choice([True, False]),
                "residual": rng.choice([True, False])}
    gated = rng.choice([True, False])
    hidden = 32 * _log(rng, 16, 448)
    rows = 32 * _log(rng, 16, 4000000 // hidden)
    return {"op": op, "tokens": _log(rng, 1, 6000), "rows": rows, "hidden": hidden, "gated": gated,
            "activation": rng.choice(["silu", "gelu_tanh"]) if gated else rng.choice(["none", "silu", "gelu_tanh"]),
            "bias": rng.choice([True, False]), "residual": rng.choice([True, False])}


def work(case):
    op, n = case["op"], case["tokens"]
    if op == "route":
        e, k = case["experts"], case["top"]
        size = 4 if case["type"] == "float32" else 2
        return {"bytes": n * (e * size + 8 * k) + 4 * e * case["bias"], "flops": 10 * n * e}
    if op == "experts":
        e, k, h, i, ranks = (case[x] for x in ("experts", "top", "hidden", "inner", "ranks"))
        met = e * (1 - (1 - k / (e * ranks)) ** n)            # experts that some token chose
        pairs = n * k / ranks
        each = 3 * i * h * 17 / 32 + case["bias"] * 2 * (2 * i + h)
        return {"bytes": met * each + n * (2 * h * (2 + case["residual"]) + 8 * k), "flops": 6 * pairs * i * h}
    h, r = case["hidden"], case["rows"]
    o = r // 2 if case["gated"] else r
    return {"bytes": r * h * 17 / 32 + 2 * n * (h + o * (1 + case["residual"])) + 2 * r * case["bias"],
            "flops": 2 * n * h * r}


# --------------------------------------------------------------- the inputs

def _randn(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32) * scale).to(torch.bfloat16)


def _activations(gen, n, h):
    """Rows as a linear layer meets them: one channel in a hundred much larger than the others."""
    x = torch.randn((n, h), generator=gen, device=DEVICE, dtype=torch.float32)
    x *= torch.where(torch.rand((h,), generator=gen, device=DEVICE) < 0.01, 20.0, 1.0)
    return x.to(torch.bfloat16)


def _checkpoint(gen, rows, h):
    """Weights as a checkpoint holds them: packed E2M1 codes [rows, h / 2], E8M0 scales [rows, h / 32]."""
    q = torch.empty((rows, h // 2), dtype=torch.uint8, device=DEVICE)
    s = torch.empty((rows, h // 32), dtype=torch.uint8, device=DEVICE)
    grid = torch.tensor(GRID, device=DEVICE)
    for a in range(0, rows, 8192):
        value, scale = _blocks(_randn(gen, min(8192, rows - a), h, scale=0.02).float())
        code = torch.bucketize(value.abs(), grid) + torch.where(value < 0, 8, 0)
        code = code.reshape(-1, h // 2, 2)
        q[a:a + 8192] = (code[..., 0] + 16 * code[..., 1]).to(torch.uint8)
        s[a:a + 8192] = (torch.frexp(scale).exponent + 126).reshape(-1, h // 32).to(torch.uint8)
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op, n = case["op"], case["tokens"]
    st = {"case": case}
    if op == "route":
        e = case["experts"]
        logits = torch.randn((n + case["padding"], e), generator=gen, device=DEVICE) * 1.5
        logits = logits.to(getattr(torch, case["type"]))
        logits[n:] = -math.inf                                # padding of a captured batch chooses nothing
        st["logits"] = logits
        st["bias"] = torch.randn((e,), generator=gen, device=DEVICE) * 0.1 if case["bias"] else None
        return st
    h = case["hidden"]
    st["x"] = _activations(gen, n, h)
    if op == "linear":
        r = case["rows"]
        out = r // 2 if case["gated"] else r
        st["w"] = _checkpoint(gen, r, h)
        st["bias"] = _randn(gen, r, scale=0.1) if case["bias"] else None
        st["residual"] = _randn(gen, n, out) if case["residual"] else None
        if own:                                               # laid out once, when the model is loaded
            import mxfp4_block_scaled_quant_amd as mx
            st["w"] = mx.mxfp4_preshuffle_weight(*st["w"], r, h)
        return st
    e, i, k, ranks = case["experts"], case["inner"], case["top"], case["ranks"]
    st["up"], st["down"] = _checkpoint(gen, e * 2 * i, h), _checkpoint(gen, e * h, i)
    st["up_bias"] = _randn(gen, e, 2 * i, scale=0.1) if case["bias"] else None
    st["down_bias"] = _randn(gen, e, h, scale=0.1) if case["bias"] else None
    st["residual"] = _randn(gen, n, h) if case["residual"] else None
    # some experts are asked for more often than others; those of other GPUs have numbers outside [0, experts)
    score = torch.randn((n, e * ranks), generator=gen, device=DEVICE)
    score = score + 0.3 * torch.randn((e * ranks,), generator=gen, device=DEVICE)
    top = torch.sort(score, descending=True, stable=True)
    st["ids"] = (top.indices[:, :k] - e * (ranks // 2)).to(torch.int32).contiguous()
    st["weights"] = torch.softmax(top.values[:, :k], 1).contiguous()
    if own:                                                   # laid out once, when the model is loaded
        import mxfp4_block_scaled_quant_amd as mx
        st["up"] = mx.MXFP4Weight(*mx.mxfp4_preshuffle_weight(*st["up"], 2 * i, h, batch=e), 2 * i, h, e)
        st["down"] = mx.MXFP4Weight(*mx.mxfp4_preshuffle_weight(*st["down"], h, i, batch=e), h, i, e)
    return st


# ---------------------------------------------------------------- the passes

def _blocks(x):
    """fp32 rows -> the E2M1 values [rows, blocks, 32] that stand for them, and the blocks' scales: a power of two
    two steps under the largest value's, the quotients rounded to nearest, ties to the even code, at most 6."""
    x = x.reshape(x.shape[0], -1, 32)
    amax = x.abs().amax(2, keepdim=True)
    exponent = (torch.frexp(amax).exponent - 3).clamp_min(-127)
    scale = torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, exponent, -127))
    v = x / scale
    m = v.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return torch.copysign((torch.round(m / step) * step).clamp_max(6.0), v), scale


def _quantised(x):
    value, scale = _blocks(x.float())
    return (value * scale).reshape(x.shape)


def _weight(q, s):
    """A checkpoint's rows as fp32."""
    code = torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1, 32).long()
    table = torch.tensor(GRID + [-g for g in GRID], device=q.device)
    scale = torch.ldexp(torch.ones(s.shape, device=s.device), s.int() - 127)
    return (table[code] * scale[..., None]).reshape(q.shape[0], -1)


def _act(v, activation):
    if activation == "silu":
        return v / (1 + torch.exp(-v))
    if activation == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _gate(v, activation, gated):
    if not gated:
        return _act(v, activation)
    half = v.shape[1] // 2
    return _act(v[:, :half], activation) * v[:, half:]


def _plain_linear(st):
    case = st["case"]
    y = _quantised(st["x"]) @ _weight(*st["w"]).t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = _gate(y, case["activation"], case["gated"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(torch.bfloat16)


def _plain_experts(st):
    case = st["case"]
    h, i = case["hidden"], case["inner"]
    x = _quantised(st["x"])
    out = torch.zeros_like(x) if st["residual"] is None else st["residual"].float()
    (uq, us), (dq, ds) = st["up"], st["down"]
    here = (st["ids"] >= 0) & (st["ids"] < case["experts"])
    for e in st["ids"][here].unique().tolist():               # the experts that some token chose
        token, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        v = x[token] @ _weight(uq[e * 2 * i:(e + 1) * 2 * i], us[e * 2 * i:(e + 1) * 2 * i]).t()
        if case["bias"]:
            v = v + st["up_bias"][e].float()
        v = _quantised(_gate(v, "silu", True).to(torch.bfloat16))
        y = v @ _weight(dq[e * h:(e + 1) * h], ds[e * h:(e + 1) * h]).t()
        if case["bias"]:
            y = y + st["down_bias"][e].float()
        out.index_add_(0, token, y * st["weights"][token, j][:, None])
    return out.to(torch.bfloat16)


def _plain_route(st):
    case = st["case"]
    k, groups = case["top"], case["groups"]
    x = st["logits"].double()
    n, e = x.shape
    open_ = x > -math.inf
    if case["scoring"] == "softmax":
        top = x.amax(1, keepdim=True)
        s = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
        s = s / s.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        s = 1 / (1 + torch.exp(-x))
    c = s + st["bias"].double() if case["bias"] else s
    c = torch.where(open_, c, -math.inf)
    if groups > 1:
        best = torch.sort(c.reshape(n, groups, -1), dim=2, descending=True).values[..., :2]
        best = torch.where(best > -math.inf, best, 0.0).sum(2)
        best = torch.where(open_.reshape(n, groups, -1).any(2), best, -math.inf)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        inside = torch.zeros((n, groups), dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        c = torch.where(inside.repeat_interleave(e // groups, 1), c, -math.inf)
    if not case["bias"]:
        x = torch.where(c > -math.inf, x, -math.inf)          # without a bias the logits' order is the scores'
        found = torch.sort(x, dim=1, descending=True, stable=True)
    else:
        found = torch.sort(c, dim=1, descending=True, stable=True)
    ids = found.indices[:, :k]
    there = found.values[:, :k] > -math.inf
    w = torch.where(there, s.gather(1, ids), 0.0)
    w = w / w.sum(1, keepdim=True).clamp_min(1e-300) * 2.5
    return w.float(), torch.where(there, ids, -1).to(torch.int32)


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"route": _plain_route, "experts": _plain_experts, "linear": _plain_linear}[op](st)
    import mxfp4_block_scaled_quant_amd as mx
    if op == "route":
        return mx.moe_route(st["logits"], case["top"], st["bias"], scoring=case["scoring"], groups=case["groups"],
                            top_groups=case["kept"], scale=2.5)
    if op == "experts":
        return mx.mxfp4_moe(st["x"], st["ids"], st["weights"], st["up"], st["down"], st["up_bias"], st["down_bias"],
                            residual=st["residual"])
    return mx.mxfp4_linear_act(st["x"], *st["w"], case["rows"], st["bias"], activation=case["activation"],
                               gated=case["gated"], residual=st["residual"])


# --------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False                                     # the checkpoint's bytes, not the library's layout
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"route": _exact_route, "experts": _exact_experts, "linear": _exact_linear}[case["op"]](st)


def _nearest(x):
    """Rows through MXFP4, in 64 bits: a code is the number of borders between neighbouring magnitudes that the
    quotient passes; a border itself goes to the even code's side."""
    x = x.double().unflatten(1, (-1, 32))
    largest = x.abs().max(2, keepdim=True).values
    power = torch.where(largest > 0, torch.floor(torch.log2(largest.clamp_min(1e-300))), -200.0)
    power = power + (torch.pow(2.0, power + 1) <= largest).double() - (torch.pow(2.0, power) > largest).double()
    unit = torch.pow(2.0, (power - 2).clamp_min(-127.0))
    a = x.abs() / unit
    code = sum((a > lim if even else a >= lim).long() for lim, even in
               ((0.25, 1), (0.75, 0), (1.25, 1), (1.75, 0), (2.5, 1), (3.5, 0), (5.0, 1)))
    return (torch.tensor(GRID, dtype=torch.float64, device=x.device)[code] * x.sign() * unit).flatten(1)


def _unpacked(q, s):
    low, high = q.bitwise_and(15).long(), q.bitwise_right_shift(4).long()
    code = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.long, device=q.device)
    code[:, 0::2], code[:, 1::2] = low, high
    value = torch.tensor(GRID, dtype=torch.float64, device=q.device)[code % 8] * (1 - 2 * (code // 8)).double()
    return value * torch.pow(2.0, s.double() - 127).repeat_interleave(32, 1)


def _activated(v, name):
    if name == "silu":
        return v * torch.special.expit(v)
    if name == "gelu_tanh":
        return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def _exact_linear(st):
    case = st["case"]
    r, half = case["rows"], case["rows"] // 2
    x = _nearest(st["x"])
    v = torch.empty((x.shape[0], r), dtype=torch.float64, device=DEVICE)
    for a in range(0, r, 4096):
        v[:, a:a + 4096] = torch.mm(x, _unpacked(*(t[a:a + 4096] for t in st["w"])).T)
    if case["bias"]:
        v += st["bias"].double()
    v = _activated(v[:, :half], case["activation"]) * v[:, half:] if case["gated"] else _activated(v, case["activation"])
    return v + st["residual"].double() if case["residual"] else v


def _exact_experts(st):
    case = st["case"]
    h, i = case["hidden"], case["inner"]
    x = _nearest(st["x"])
    out = torch.zeros_like(x)
    for e in range(case["experts"]):
        share = torch.where(st["ids"] == e, st["weights"], 0.0).double().sum(1)
        token = torch.nonzero((st["ids"] == e).any(1))[:, 0]
        if not len(token):
            continue
        up = slice(e * 2 * i, (e + 1) * 2 * i)
        v = torch.mm(x[token], _unpacked(st["up"][0][up], st["up"][1][up]).T)
        v = v + st["up_bias"][e].double() if case["bias"] else v
        v = _nearest((_activated(v[:, :i], "silu") * v[:, i:]).to(torch.bfloat16))      # held in bf16, then quantised
        down = slice(e * h, (e + 1) * h)
        y = torch.mm(v, _unpacked(st["down"][0][down], st["down"][1][down]).T)
        y = y + st["down_bias"][e].double() if case["bias"] else y
        out[token] += y * share[token, None]
    return out + st["residual"].double() if case["residual"] else out


def _exact_route(st):
    case = st["case"]
    k, groups, e = case["top"], case["groups"], case["experts"]
    bias = st["bias"].double() if case["bias"] else None
    weights, ids = [], []

    def place(c):
        """Each value's place in its row, the largest first, equal ones by index."""
        first, then = c[:, :, None], c[:, None, :]
        at = torch.arange(c.shape[1], device=c.device)
        return ((then > first) | ((then == first) & (at[None, :] < at[:, None]))).sum(2)

    for part in st["logits"].double().split(512):
        s = torch.softmax(part, 1) if case["scoring"] == "softmax" else torch.special.expit(part)
        s = torch.where(part.isinf(), 0.0, s)
        c = s if bias is None else s + bias
        c = c.masked_fill(part.isinf(), -math.inf)
        if groups > 1:
            each = c.unflatten(1, (groups, -1))
            two = each.topk(2, 2).values
            total = two.masked_fill(two.isinf(), 0.0).sum(2).masked_fill(two[..., 0].isinf(), -math.inf)
            chosen = place(total) < case["kept"]
            c = c.masked_fill(~chosen[:, :, None].expand_as(each).flatten(1), -math.inf)
        order = place(c if bias is not None else part.masked_fill(c.isinf(), -math.inf))
        one_hot = torch.zeros((len(part), e, k), dtype=torch.float64, device=part.device)
        for j in range(k):
            one_hot[:, :, j] = ((order == j) & ~c.isinf()).double()
        w = (s[:, :, None] * one_hot).sum(1)
        total = w.sum(1, keepdim=True)
        weights.append(torch.where(total > 0, 2.5 * w / total, 0.0))
        at = torch.arange(e, device=part.device, dtype=torch.float64)
        ids.append(((at[:, None] * one_hot).sum(1) - (one_hot.sum(1) == 0).double()).to(torch.int32))
    return torch.cat(weights), torch.cat(ids)
