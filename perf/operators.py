"""Cases of the latent-attention operators, and their plain forms.

Four operators of a serving step with one shared latent vector a token:

* ``append``   the latent's norm, the position rotation of the key and query
               parts, and the write into the paged cache
* ``decode``   attention of a few query tokens a request over the paged
               latents themselves (absorbed form)
* ``prefix``   the same, where all requests share one long prefix
* ``prefill``  causal attention of whole prompts or chunks over keys and
               values expanded per head (expanded form)

``own`` chooses what :func:`run` does: the plain form in torch's elementary
operations, or the calls of :mod:`mxfp4_block_scaled_quant_amd`.
"""

import math
import random

import torch

own = False

LATENT, ROPE = 512, 64          # the cached row: normed latent, rotated key part
DEVICE = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the first tokens of one conversation: nothing but latency
        {"name": "decode_one_short", "op": "decode", "batch": 1, "tokens": 1, "heads": 16, "low": 777, "high": 777,
         "page": 64},
        # a few long documents, each spread over many compute units
        {"name": "decode_few_long", "op": "decode", "batch": 6, "tokens": 1, "heads": 16, "low": 40001, "high": 65531,
         "page": 16},
        # a full serving batch of unequal conversations
        {"name": "decode_many_ragged", "op": "decode", "batch": 128, "tokens": 1, "heads": 16, "low": 1, "high": 16000,
         "page": 64},
        # drafted tokens checked together, all heads on one GPU: the matrix units' side
        {"name": "decode_drafted_all_heads", "op": "decode", "batch": 12, "tokens": 4, "heads": 128, "low": 1500,
         "high": 8191, "page": 64},
        # several samples of one short prompt
        {"name": "prefix_samples", "op": "prefix", "batch": 8, "tokens": 1, "heads": 16, "prefix": 1021, "low": 1,
         "high": 60, "page": 16},
        # a serving batch under one long system prompt
        {"name": "prefix_system_prompt", "op": "prefix", "batch": 96, "tokens": 1, "heads": 16, "prefix": 24571,
         "low": 5, "high": 900, "page": 64},
        # one short prompt
        {"name": "prefill_short", "op": "prefill", "heads": 16, "nope": 128, "value": 128, "batch": 1, "low": 333,
         "high": 333, "past": 0},
        # prompts of unequal lengths in one batch
        {"name": "prefill_ragged", "op": "prefill", "heads": 16, "nope": 192, "value": 256, "batch": 9, "low": 17,
         "high": 4001, "past": 0},
        # a chunk of a long prompt, over what came before it
        {"name": "prefill_chunk", "op": "prefill", "heads": 16, "nope": 128, "value": 128, "batch": 2, "low": 1900,
         "high": 2048, "past": 14003},
        # one long document
        {"name": "prefill_long", "op": "prefill", "heads": 16, "nope": 192, "value": 256, "batch": 1, "low": 16384,
         "high": 16384, "past": 0},
        # one decoding step's new tokens, a few of them padding of a captured batch
        {"name": "append_step", "op": "append", "heads": 16, "nope": 192, "count": 61, "padding": 3, "page": 64,
         "interleaved": True},
        # a prompt's tokens
        {"name": "append_prompt", "op": "append", "heads": 16, "nope": 192, "count": 16001, "padding": 0, "page": 64,
         "interleaved": False},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefix", "prefill", "prefill", "append"])
    if op == "append":
        return {"op": op, "heads": rng.choice([1, 5, 8, 16, 32]), "nope": rng.choice([128, 192]),
                "count": _log(rng, 1, 8000), "padding": rng.choice([0, 0, 2, 7]),
                "page": rng.choice([1, 16, 48, 64, 128]), "interleaved": rng.choice([True, False])}
    if op == "prefill":
        nope, value = rng.choice([(128, 128), (192, 256)])
        batch = rng.choice([1, 1, 2, 3, 7, 20])
        high = _log(rng, 1, 9000 // batch)
        past = rng.choice([0, 0, _log(rng, 1, 6000)])
        return {"op": op, "heads": rng.choice([1, 3, 8, 16]), "nope": nope, "value": value, "batch": batch,
                "low": rng.randint(1, high), "high": high, "past": past}
    heads = rng.choice([1, 5, 8, 16, 16, 20, 32, 64, 128])
    tokens = rng.choice([1, 1, 1, 2, 3, 4])
    page = rng.choice([1, 16, 48, 64, 128])
    batch = _log(rng, 1, 128)
    if op == "prefix":
        prefix = _log(rng, 50, max(60, min(20000, 30000000 // (batch * tokens * heads))))
        high = _log(rng, tokens, 1000)
        return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "prefix": prefix,
                "low": rng.randint(tokens, high), "high": high, "page": page}
    high = _log(rng, tokens, max(16, min(100000, 800000 // batch, 40000000 // (batch * tokens * heads))))
    return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "low": rng.randint(tokens, high),
            "high": high, "page": page}


def _lengths(case):
    """The requests' lengths: part of the case, not of the seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = [rng.randint(case["low"], case["high"]) for _ in range(case["batch"])]
    n[0] = case["high"]
    n[-1] = case["low"] if case["batch"] > 1 else n[-1]
    return n


def work(case):
    op = case["op"]
    row = LATENT + ROPE
    if op == "append":
        n = case["count"]
        # each token: its latent row in and out, its heads' rotated part in and
        # out, its angles, its slot and position
        return {"bytes": n * (4 * row + 4 * case["heads"] * ROPE + 4 * ROPE + 16) + 2 * LATENT,
                "flops": n * (4 * LATENT + 3 * ROPE * (1 + case["heads"]))}
    lens = _lengths(case)
    h = case["heads"]
    if op == "prefill":
        d, v, past = case["nope"] + ROPE, case["value"], case["past"]
        pairs = sum(n * past + n * (n + 1) // 2 for n in lens)
        keys = sum(n + past for n in lens)
        return {"bytes": 2 * (sum(lens) * h * (d + v) + keys * (h * (case["nope"] + v) + ROPE)) + 4 * sum(lens) * h,
                "flops": 2 * h * pairs * (d + v)}
    s, prefix = case["tokens"], case.get("prefix", 0)
    pairs = sum(s * n - s * (s - 1) // 2 for n in lens) + prefix * s * len(lens)
    rows = len(lens) * s * h
    return {"bytes": 2 * row * (sum(lens) + prefix) + rows * (2 * row + 2 * LATENT + 4),
            "flops": 2 * h * pairs * (row + LATENT)}


# --------------------------------------------------------------- the inputs

def _randn(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32) * scale).to(torch.bfloat16)


def _pages(rng, lens, page):
    """Page numbers of each request, in no order, and how many pages there are."""
    need = [-(-n // page) for n in lens]
    ids = list(range(sum(need) + 3))
    rng.shuffle(ids)
    tables, at = [], 0
    for n in need:
        tables.append(ids[at:at + n])
        at += n
    return tables, len(ids)


def _table(tables):
    width = max(1, max(len(t) for t in tables))
    return torch.tensor([t + [0] * (width - len(t)) for t in tables], dtype=torch.int32, device=DEVICE)


def _angles(positions):
    """cos and sin of every position's angles, [positions, 2 * 32] fp32."""
    freq = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=DEVICE) / ROPE)
    a = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    rng = random.Random(seed)
    op = case["op"]
    st = {"case": case}
    if op == "append":
        n, pad, h = case["count"], case["padding"], case["heads"]
        pages = -(-n // case["page"]) + 2
        slots = rng.sample(range(pages * case["page"]), n)
        row = list(range(n + pad))
        rng.shuffle(row)
        row = sorted(row[:n])                         # the rows that are no padding
        slot = torch.full((n + pad,), -1, dtype=torch.int64)
        slot[torch.tensor(row)] = torch.tensor(slots)
        st["row"] = torch.tensor(row, device=DEVICE)
        st["slots"] = slot.to(DEVICE)
        limit = 32768
        st["positions"] = torch.randint(0, limit, (n + pad,), generator=gen, device=DEVICE)
        st["cos_sin"] = _angles(limit)
        st["kv"] = _randn(gen, n + pad, LATENT + ROPE)
        st["weight"] = _randn(gen, LATENT, scale=0.2) + 1
        st["cache"] = _randn(gen, pages, case["page"], LATENT + ROPE)
        # the query projection's output, and the absorbed query that takes its rotated part
        st["q"] = _randn(gen, n + pad, h, case["nope"] + ROPE)
        st["q_absorbed"] = _randn(gen, n + pad, h, LATENT + ROPE)
        return st
    lens = _lengths(case)
    st["lens"] = lens
    if op == "prefill":
        h, past = case["heads"], case["past"]
        keys = [n + past for n in lens]
        d = case["nope"] + ROPE
        st["keys"] = keys
        st["q"] = _randn(gen, sum(lens), h, d)
        st["k_nope"] = _randn(gen, sum(keys), h, case["nope"])
        st["k_pe"] = _randn(gen, sum(keys), ROPE)
        st["v"] = _randn(gen, sum(keys), h, case["value"])
        st["cu_q"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEVICE)
        st["cu_k"] = torch.tensor([sum(keys[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEVICE)
        st["scale"] = 1.5 / math.sqrt(d)
        return st
    every = lens + [case["prefix"]] if op == "prefix" else lens
    tables, pages = _pages(rng, every, case["page"])
    st["cache"] = _randn(gen, pages, case["page"], LATENT + ROPE)
    st["q"] = _randn(gen, case["batch"], case["tokens"], case["heads"], LATENT + ROPE)
    st["scale"] = 1.0 / 16.0
    if op == "prefix":
        st["prefix_table"] = torch.tensor(tables.pop(), dtype=torch.int32, device=DEVICE)
    st["table"] = _table(tables)
    st["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    return st


# ---------------------------------------------------------------- the passes

def _softmax_product(s, v, visible):
    """Softmax of the scores s [..., keys] where visible, times v [keys, n],
    and the scores' log-sum-exp."""
    s = s.masked_fill(~visible, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total, (m + torch.log(total)).squeeze(-1)


def _rows_of(cache, table, n):
    """The first n cached rows of a page table, fp32."""
    page = cache.shape[1]
    return cache[table[:-(-n // page)].long()].reshape(-1, LATENT + ROPE)[:n].float()


def _plain_decode(st):
    q, lens, case = st["q"], st["lens"], st["case"]
    b, s, h, _ = q.shape
    prefix = case.get("prefix", 0)
    shared = _rows_of(st["cache"], st["prefix_table"], prefix) if prefix else None
    out = torch.empty((b, s, h, LATENT), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((b, s, h), dtype=torch.float32, device=q.device)
    for i, n in enumerate(lens):
        kv = _rows_of(st["cache"], st["table"][i], n)
        if prefix:
            kv = torch.cat([shared, kv])
        at = torch.arange(n + prefix, device=q.device)
        last = n + prefix - s + torch.arange(s, device=q.device)      # the last key each token sees
        visible = (at[None, :] <= last[:, None])[:, None, :].expand(s, h, -1).reshape(s * h, -1)
        scores = (q[i].float().reshape(s * h, -1) @ kv.t()) * st["scale"]
        o, e = _softmax_product(scores, kv[:, :LATENT], visible)
        out[i] = o.reshape(s, h, LATENT).to(torch.bfloat16)
        lse[i] = e.reshape(s, h)
    return out, lse


def _plain_prefill(st):
    q, case = st["q"], st["case"]
    t, h, _ = q.shape
    out = torch.empty((t, h, case["value"]), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((t, h), dtype=torch.float32, device=q.device)
    tq = tk = 0
    for n, keys in zip(st["lens"], st["keys"]):
        visible = (torch.arange(keys, device=q.device)[None, :]
                   <= (keys - n + torch.arange(n, device=q.device))[:, None])
        pe = st["k_pe"][tk:tk + keys].float()
        for i in range(h):
            k = torch.cat([st["k_nope"][tk:tk + keys, i].float(), pe], 1)
            scores = (q[tq:tq + n, i].float() @ k.t()) * st["scale"]
            o, e = _softmax_product(scores, st["v"][tk:tk + keys, i].float(), visible)
            out[tq:tq + n, i] = o.to(torch.bfloat16)
            lse[tq:tq + n, i] = e
        tq, tk = tq + n, tk + keys
    return out, lse


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(st):
    case = st["case"]
    angle = st["cos_sin"][st["positions"]]
    cos, sin = angle[:, :ROPE // 2], angle[:, ROPE // 2:]
    x = st["kv"].float()
    c = x[:, :LATENT]
    c = c * torch.rsqrt((c * c).sum(1, keepdim=True) / LATENT + 1e-6) * st["weight"].float()
    rows = torch.cat([c, _rotate(x[:, LATENT:], cos, sin, case["interleaved"])], 1).to(torch.bfloat16)
    keep = st["row"]
    st["cache"].view(-1, LATENT + ROPE)[st["slots"][keep]] = rows[keep]
    q = st["q"][..., case["nope"]:].float()
    st["q_absorbed"][..., LATENT:] = _rotate(q, cos[:, None], sin[:, None], case["interleaved"]).to(torch.bfloat16)
    return st["cache"], st["q_absorbed"]


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"append": _plain_append, "prefill": _plain_prefill}.get(op, _plain_decode)(st)
    import mxfp4_block_scaled_quant_amd as mx
    if op == "append":
        mx.mla_cache_append(st["kv"], st["weight"], st["cache"], st["slots"], st["positions"], st["cos_sin"],
                            q_pe=st["q"][..., case["nope"]:], q_out=st["q_absorbed"][..., LATENT:], eps=1e-6,
                            interleaved=case["interleaved"])
        return st["cache"], st["q_absorbed"]
    if op == "prefill":
        return mx.mla_prefill(st["q"], st["k_nope"], st["k_pe"], st["v"], st["cu_q"], st["cu_k"], st["scale"],
                              return_lse=True)
    if op == "prefix":
        return mx.mla_decode_shared_prefix(st["q"], st["cache"], st["prefix_table"], case["prefix"], st["table"],
                                           st["lengths"], st["scale"], return_lse=True)
    return mx.mla_decode(st["q"], st["cache"], st["table"], st["lengths"], st["scale"], return_lse=True)


# --------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(st)
    if op == "prefill":
        h, d = st["q"].shape[1:]
        out = torch.empty((st["q"].shape[0], h, case["value"]), dtype=torch.float64, device=DEVICE)
        lse = torch.empty(out.shape[:2], dtype=torch.float64, device=DEVICE)
        cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
        for i in range(case["batch"]):
            n, keys = cq[i + 1] - cq[i], ck[i + 1] - ck[i]
            for j in range(h):
                k = torch.empty((keys, d), dtype=torch.float64, device=DEVICE)
                k[:, :case["nope"]] = st["k_nope"][ck[i]:ck[i + 1], j]
                k[:, case["nope"]:] = st["k_pe"][ck[i]:ck[i + 1]]
                v = st["v"][ck[i]:ck[i + 1], j].double()
                for a in range(0, n, 4096):
                    b = min(n, a + 4096)
                    hi = keys - n + b                     # no row of this block sees a later key
                    z = torch.mm(st["q"][cq[i] + a:cq[i] + b, j].double(), k[:hi].T) * st["scale"]
                    z += torch.full_like(z, -math.inf).triu(keys - n + a + 1)
                    e = torch.logsumexp(z, 1)
                    out[cq[i] + a:cq[i] + b, j] = torch.mm(torch.exp(z - e[:, None]), v[:hi])
                    lse[cq[i] + a:cq[i] + b, j] = e
        return out, lse
    b, s, h, _ = st["q"].shape
    out = torch.empty((b, s, h, LATENT), dtype=torch.float64, device=DEVICE)
    lse = torch.empty((b, s, h), dtype=torch.float64, device=DEVICE)
    page = case["page"]
    flat = st["cache"].reshape(-1, LATENT + ROPE)
    for i in range(b):
        n = int(st["lengths"][i])
        t = torch.arange(n, device=DEVICE)
        slots = st["table"][i].long()[t // page] * page + t % page
        if op == "prefix":
            u = torch.arange(case["prefix"], device=DEVICE)
            slots = torch.cat([st["prefix_table"].long()[u // page] * page + u % page, slots])
        kv = flat[slots].double()
        for j in range(s):
            seen = kv[:len(slots) - (s - 1 - j)]
            z = torch.mm(st["q"][i, j].double(), seen.T) * st["scale"]
            lse[i, j] = torch.logsumexp(z, 1)
            out[i, j] = torch.mm(torch.softmax(z, 1), seen[:, :LATENT])
    return out, lse


def _exact_append(st):
    case = st["case"]
    cache, q_out = st["cache"].double(), st["q_absorbed"].double()
    half = ROPE // 2
    table = st["cos_sin"].double()[st["positions"]]
    turn = torch.complex(table[:, :half], table[:, half:])

    def rotated(x, by):
        pairs = x.unflatten(-1, (half, 2)) if case["interleaved"] else x.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * by
        both = torch.stack([z.real, z.imag], -1 if case["interleaved"] else -2)
        return both.flatten(-2)

    x = st["kv"].double()
    latent = x[:, :LATENT]
    norm = latent / torch.sqrt(latent.square().mean(1, keepdim=True) + 1e-6) * st["weight"].double()
    rows = torch.cat([norm, rotated(x[:, LATENT:], turn)], 1)
    for_cache = cache.view(-1, LATENT + ROPE)
    written = st["slots"] >= 0
    for_cache[st["slots"][written]] = rows[written]
    q_out[..., LATENT:] = rotated(st["q"][..., case["nope"]:].double(), turn[:, None])
    return cache, q_out
