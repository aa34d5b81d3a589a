"""Attention over a paged cache, from the projections' rows to the output projection's, each operator
in a plain torch form and as calls of libtb.so.

Three operators, those of a full-attention layer between its two projections, measured on cases from
one decoded token, where latency counts, to long prompts:

  kvplan  block tables and slot maps of a step from the requests' lengths: pages of ended requests go
          back to the free list, new pages are taken from it, and every new token gets its position
          and its slot (once a step, for all layers)
  rope    rotary positions on strided rows of a fused projection (interleaved or half layout, part of
          the head, scaled for long contexts); keys and values go into the pages of the cache
  attn    attention of each request's new tokens over its pages (one token while decoding, a chunk of
          a prompt, both in one batch), causal, optionally within a window, with the output gate of
          the fused projection

A case names its operator in "op". Head counts and widths are those of the fused projection of 9216
rows (16 query heads, 2 key-value heads of 256, a gate as wide as the query), and generic ones.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
I32 = torch.int32
HALF, INTERLEAVED = "half", "interleaved"


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one request decodes one token
        {"name": "kvplan-1", "op": "kvplan", "requests": 1, "context": 4096, "chunk": 1, "rows": 1, "page": 16},
        # a server's step: 250 requests, most decode, some bring a chunk of their prompt, some have ended
        {"name": "kvplan-250", "op": "kvplan", "requests": 250, "context": 16384, "chunk": 509, "rows": 2048, "page": 16},
        # the largest step: 2048 requests, 16384 rows
        {"name": "kvplan-2048", "op": "kvplan", "requests": 2048, "context": 8192, "chunk": 1024, "rows": 16384, "page": 16},
        # one decoded token's fused projection row in fp32 (what the ternary products write), a quarter of each head rotated
        {"name": "rope-1", "op": "rope", "tokens": 1, "heads": 16, "kv": 2, "dim": 256, "rot": 64, "layout": HALF, "rows": "f32", "q": "f32",
         "cache": "bf16", "page": 16, "far": 4096, "stretch": 1.0, "gate": True, "pad": 0},
        # 33 decodes in a batch padded to 37 rows, interleaved pairs, the whole head
        {"name": "rope-37", "op": "rope", "tokens": 37, "heads": 24, "kv": 8, "dim": 128, "rot": 128, "layout": INTERLEAVED, "rows": "f16", "q": "f16",
         "cache": "f16", "page": 32, "far": 32768, "stretch": 1.0, "gate": False, "pad": 4},
        # an odd chunk far into a long context, fp32 rows, q in the cache's type
        {"name": "rope-509", "op": "rope", "tokens": 509, "heads": 16, "kv": 2, "dim": 256, "rot": 64, "layout": HALF, "rows": "f32", "q": "bf16",
         "cache": "bf16", "page": 16, "far": 1000000, "stretch": 8.0, "gate": True, "pad": 0},
        # a prefill of 8192 tokens
        {"name": "rope-8192", "op": "rope", "tokens": 8192, "heads": 16, "kv": 2, "dim": 256, "rot": 256, "layout": HALF, "rows": "bf16", "q": "bf16",
         "cache": "bf16", "page": 64, "far": 131072, "stretch": 4.0, "gate": True, "pad": 0},
        # one decoded token over 4096 cached ones, fp32 rows to feed the ternary output projection
        {"name": "attn-1", "op": "attn", "requests": 1, "chunk": 1, "context": 4096, "heads": 16, "kv": 2, "dim": 256, "rows": "f32", "cache": "bf16",
         "page": 16, "window": 0, "gate": True, "ragged": False},
        # one decoded token at the end of a long document
        {"name": "attn-1-long", "op": "attn", "requests": 1, "chunk": 1, "context": 131072, "heads": 16, "kv": 2, "dim": 256, "rows": "f32",
         "cache": "bf16", "page": 64, "window": 0, "gate": True, "ragged": False},
        # 48 concurrent decodes of contexts up to 16384
        {"name": "attn-48", "op": "attn", "requests": 48, "chunk": 1, "context": 16384, "heads": 16, "kv": 2, "dim": 256, "rows": "bf16",
         "cache": "bf16", "page": 16, "window": 0, "gate": True, "ragged": True},
        # a mixed step: some requests decode, others bring chunks of up to 509 tokens; a window of 1024
        {"name": "attn-mixed", "op": "attn", "requests": 12, "chunk": 509, "context": 4096, "heads": 24, "kv": 8, "dim": 128, "rows": "f16",
         "cache": "f16", "page": 32, "window": 1024, "gate": False, "ragged": True},
        # a prompt's chunk of 2048 tokens behind 8192 cached ones
        {"name": "attn-2048", "op": "attn", "requests": 1, "chunk": 2048, "context": 8192, "heads": 16, "kv": 2, "dim": 256, "rows": "bf16",
         "cache": "bf16", "page": 64, "window": 0, "gate": True, "ragged": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["kvplan", "rope", "attn", "attn"])
    if op == "kvplan":
        requests = _log(rng, 1, 2048)
        return {"op": op, "requests": requests, "context": _log(rng, 1, 8192), "chunk": _log(rng, 1, 1024),
                "rows": _log(rng, requests, min(16384, requests * 64)), "page": rng.choice([16, 32, 64, 128])}
    heads, kv = rng.choice([(16, 2), (16, 2), (24, 8), (8, 8), (5, 1), (12, 4), (32, 4)])
    dim, page = rng.choice([64, 128, 256, 256]), rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "bf16", "f16"])
    if op == "rope":
        rows = rng.choice([cache, "f32"])
        tokens = _log(rng, 1, 8192 * 16 * 256 // (heads * dim) // (SIZE[rows] // 2) // 2)
        return {"op": op, "tokens": tokens, "heads": heads, "kv": kv, "dim": dim, "rot": dim // rng.choice([1, 1, 2, 4]),
                "layout": rng.choice([HALF, INTERLEAVED]), "rows": rows, "q": rng.choice([cache, "f32"]) if rows == "f32" else cache,
                "cache": cache, "page": page, "far": _log(rng, 64, 1000000), "stretch": rng.choice([1.0, 4.0, 8.0]),
                "gate": rng.random() < 0.5, "pad": rng.choice([0, 0, 3]) if tokens > 8 else 0}
    rows = rng.choice([cache, cache, "f32"])
    requests = _log(rng, 1, 64)
    chunk = 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
    context = _log(rng, 1, 131072)
    window = rng.choice([0, 0, 0, 128, 4096])
    while _flops(requests, chunk, context, heads, dim) > (1.2e11 if rows == "f32" else 1.5e11) or requests * (chunk + context) * kv * dim > 134_000_000:
        if requests > 1 and requests * 64 > context:
            requests = (requests + 1) // 2
        elif chunk > context or context < 512:
            chunk = (chunk + 1) // 2
        else:
            context //= 2
    return {"op": op, "requests": requests, "chunk": chunk, "context": context, "heads": heads, "kv": kv, "dim": dim, "rows": rows, "cache": cache,
            "page": page, "window": window, "gate": rng.random() < 0.5, "ragged": requests > 1}


def _flops(requests, chunk, context, heads, dim):
    return 4 * requests * chunk * (context + chunk) * heads * dim


# ---------------------------------------------------------------------------------------------
# Inputs, and the buffers that a user's program keeps
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def _ints(v):
    return torch.tensor(v, dtype=I32, device=DEV)


def _lengths(c):
    """(cached, new) tokens of each request: a case always has the same."""
    rng = random.Random("%s %s %s %s" % (c["op"], c["requests"], c["context"], c["chunk"]))
    got = []
    for i in range(c["requests"]):
        if c["op"] == "attn":
            context = c["context"] if not c["ragged"] or i == 0 else _log(rng, 1, c["context"])
            got.append((context, c["chunk"] if not c["ragged"] or i % 3 == 0 else 1 if i % 3 == 1 else _log(rng, 1, c["chunk"])))
        else:
            context = c["context"] if i == 0 else _log(rng, 1, c["context"])
            kind = rng.random()
            # decodes, a chunk of a prompt, has ended (-1), waits
            got.append((context, 1 if i == 0 or kind < 0.8 else _log(rng, 1, c["chunk"]) if kind < 0.9 else -1 if kind < 0.97 else 0))
    return got


def _prepare_kvplan(c, g):
    page, pairs = c["page"], _lengths(c)
    # the cache's pages in the order in which they have come free; each request holds those of its context
    held = [-(-context // page) for context, _ in pairs]
    width = -(-(c["context"] + c["chunk"]) // page)
    pages = sum(held) + -(-c["rows"] // page) + 2 * len(pairs) + 64
    order = torch.randperm(pages, generator=g, device=DEV).to(I32)
    n = torch.tensor(held, device=DEV)
    at = torch.arange(width, device=DEV)
    first = (n.cumsum(0) - n)[:, None]
    table = torch.where(at < n[:, None], order[(first + at).clamp(max=pages - 1)], -1).to(I32).contiguous()
    free = torch.full((pages,), -1, dtype=I32, device=DEV)
    left = pages - sum(held)
    free[:left] = order[sum(held):]
    s, r = len(pairs), c["rows"]
    return {"context": _ints([a for a, _ in pairs]), "fresh": _ints([b for _, b in pairs]), "page": page, "pages": pages, "table": table,
            "free": free, "count": _ints([left]), "lengths": _empty(s, dtype=I32), "offsets": _empty(s + 1, dtype=I32),
            "positions": _empty(r, dtype=I32), "slots": _empty(r, dtype=I32), "left": _empty(1, dtype=I32), "missing": _empty(1, dtype=I32)}


def _frequencies(rot, stretch, base=1000000.0, trained=32768.0):
    """Radians per position of each pair, in 64 bits, and the factor on the rotated part. stretch > 1: pairs that turn less than
    once over the trained length are slowed by it, those that turn 32 times are kept, those between are mixed."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if stretch <= 1:
        return f, 1.0
    keep = ((trained * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
    return f * (keep + (1 - keep) / stretch), 0.1 * math.log(stretch) + 1


def _prepare_rope(c, g):
    t, heads, kv, dim, page = c["tokens"], c["heads"], c["kv"], c["dim"], c["page"]
    # rows of the fused projection: query, gate (if the model has one), key, value
    width = heads * dim * (2 if c["gate"] else 1)
    fused = torch.randn(t, width + 2 * kv * dim, generator=g, device=DEV).to(TYPES[c["rows"]])
    freq, factor = _frequencies(c["rot"], c["stretch"])
    pages = -(-t // page) + 1
    place = torch.randperm(pages, generator=g, device=DEV)
    i = torch.arange(t, device=DEV)
    real = i < t - c["pad"]
    positions = torch.where(real, c["far"] - t + i if c["far"] >= t else i, -1)
    # a request's tokens fill page after page, wherever these lie
    slots = torch.where(real, place[i // page] * page + i % page, -1)
    cache = TYPES[c["cache"]]
    return {"fused": fused, "q": fused[:, :heads * dim].view(t, heads, dim), "k": fused[:, width:width + kv * dim].view(t, kv, dim),
            "v": fused[:, width + kv * dim:].view(t, kv, dim), "freq": freq.to(DEV), "factor": factor, "layout": c["layout"], "rot": c["rot"],
            "positions": positions.to(I32), "slots": slots.to(I32), "page": page,
            "kcache": torch.zeros(pages, kv, page, dim, dtype=cache, device=DEV), "vcache": torch.zeros(pages, kv, page, dim, dtype=cache, device=DEV),
            "out": torch.zeros(t, heads, dim, dtype=TYPES[c["q"]], device=DEV)}


def _prepare_attn(c, g):
    heads, kv, dim, page = c["heads"], c["kv"], c["dim"], c["page"]
    pairs = _lengths(c)
    lengths = [a + b for a, b in pairs]
    held = [-(-n // page) for n in lengths]
    pages = sum(held)
    order = torch.randperm(pages, generator=g, device=DEV).to(I32)
    n = torch.tensor(held, device=DEV)
    at = torch.arange(max(held), device=DEV)
    table = torch.where(at < n[:, None], order[((n.cumsum(0) - n)[:, None] + at).clamp(max=pages - 1)], -1).to(I32).contiguous()
    offsets = [0]
    for _, new in pairs:
        offsets.append(offsets[-1] + new)
    t, cache, rows = offsets[-1], TYPES[c["cache"]], TYPES[c["rows"]]
    kc = torch.randn(pages, kv, page, dim, generator=g, device=DEV, dtype=cache)
    # some channels of the keys are larger than the others, and scores spread over several units
    kc *= torch.where(torch.rand(dim, generator=g, device=DEV) < 0.03, 4.0, 1.0).to(cache)
    vc = torch.randn(pages, kv, page, dim, generator=g, device=DEV, dtype=cache)
    q = torch.randn(t, heads, dim, generator=g, device=DEV).to(rows)
    s = {"q": q, "kcache": kc, "vcache": vc, "table": table, "offsets": _ints(offsets), "lengths": _ints(lengths), "page": page,
         "scale": 1.0 / math.sqrt(dim), "window": c["window"], "gate": None, "chunk": max(b for _, b in pairs), "longest": max(lengths),
         # scratch that the program keeps for every layer
         "ws": _empty(192 << 20, dtype=torch.uint8), "out": _empty(t, heads, dim, dtype=rows)}
    if c["gate"]:  # within the rows of the fused projection
        fused = torch.randn(t, 2 * (heads + kv) * dim, generator=g, device=DEV).to(rows)
        s["gate"] = fused[:, heads * dim:2 * heads * dim].view(t, heads, dim)
    return s


_PREPARE = {"kvplan": _prepare_kvplan, "rope": _prepare_rope, "attn": _prepare_attn}


def prepare(case, seed):
    state = _PREPARE[case["op"]](case, _gen(seed))
    state["op"] = case["op"]
    return state


# ---------------------------------------------------------------------------------------------
# Plain forms, in 32 bits (angles in 64)
# ---------------------------------------------------------------------------------------------
def _plain_kvplan(s):
    page, pages, table = s["page"], s["pages"], s["table"].long()
    requests, width = table.shape
    context, fresh = s["context"].long().clamp(min=0), s["fresh"].long()
    at = torch.arange(width, device=DEV)
    # pages of ended requests are pushed on the free list
    ended = fresh < 0
    have = ((context + page - 1) // page).clamp(max=width)
    back = table[ended[:, None] & (at < have[:, None]) & (table >= 0) & (table < pages)]
    free, count = s["free"].long(), s["count"].long()
    free = free.scatter(0, count + torch.arange(back.numel(), device=DEV), back)
    count = count + back.numel()
    # new tokens, as far as there are rows
    rows = s["positions"].numel()
    offsets = torch.cat((torch.zeros_like(count), fresh.clamp(min=0).cumsum(0))).clamp(max=rows)
    new = offsets[1:] - offsets[:-1]
    lengths = torch.where(ended, 0, context + new)
    # new pages are popped from its end, request by request
    need = ((lengths + page - 1) // page).clamp(max=width)
    take = (need - have).clamp(min=0)
    rank = (take.cumsum(0) - take)[:, None] + at - have[:, None]
    taken = (at >= have[:, None]) & (at < need[:, None])
    place = count - 1 - rank
    table = torch.where(taken, torch.where(place >= 0, free[place.clamp(0, pages - 1)], -1), table)
    left = (count - take.sum()).clamp(min=0)
    # each row's position and slot
    row = torch.arange(rows, device=DEV)
    r = torch.searchsorted(offsets[1:].contiguous(), row, right=True).clamp(max=requests - 1)
    real = row < offsets[-1]
    position = torch.where(real, lengths[r] - new[r] + row - offsets[r], -1)
    index = position // page
    entry = table[r, index.clamp(0, width - 1)]
    placed = real & (index < width) & (entry >= 0) & (entry < pages)
    slot = torch.where(placed, entry * page + position % page, -1)
    missing = (real & ~placed).sum()[None]
    return {k: v.to(I32) for k, v in {"table": table, "free": free, "left": left, "lengths": lengths, "offsets": offsets, "positions": position,
                                      "slots": slot, "missing": missing}.items()}


def _plain_turn(x, cos, sin, rot, layout):
    """Rows x [tokens][heads][dim], the pairs of their first `rot` elements turned, in fp32."""
    x = x.float()
    cos, sin = cos[:, None], sin[:, None]
    if layout == HALF:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["factor"]).float() for f in (torch.cos, torch.sin))
    q, k = (_plain_turn(s[n], cos, sin, s["rot"], s["layout"]) for n in ("q", "k"))
    kc, vc, page = s["kcache"], s["vcache"], s["page"]
    slot = s["slots"].long()
    kept = slot >= 0
    slot = slot[kept]
    kc[slot // page, :, slot % page] = k[kept].to(kc.dtype)
    vc[slot // page, :, slot % page] = s["v"][kept].to(vc.dtype)
    real = (s["positions"] >= 0)[:, None, None]
    return {"q": torch.where(real, q, 0.0).to(s["out"].dtype), "k": kc, "v": vc}


def _plain_attn(s):
    page, q = s["page"], s["q"]
    heads, dim = q.shape[1:]
    kv = s["kcache"].shape[1]
    offsets, lengths = s["offsets"].long(), s["lengths"].long()
    new = offsets[1:] - offsets[:-1]
    # each request's rows padded to the longest chunk, its keys to the longest request
    i, key = torch.arange(s["chunk"], device=DEV), torch.arange(s["longest"], device=DEV)
    real = i < new[:, None]
    row = torch.where(real, offsets[:-1, None] + i, 0)
    position = (lengths - new)[:, None] + i
    x = q[row].float().view(*row.shape, kv, heads // kv, dim).permute(0, 2, 3, 1, 4)
    pages = s["table"].long()[:, key // page].clamp(min=0)
    k, v = (s[n][pages, :, key % page].float().transpose(1, 2).unsqueeze(2) for n in ("kcache", "vcache"))
    seen = (key <= position[..., None]) & (key < lengths[:, None, None])
    if s["window"]:
        seen &= key > position[..., None] - s["window"]
    score = torch.matmul(x.reshape(*x.shape[:2], 1, -1, dim), k.transpose(-1, -2).contiguous()).view(*x.shape[:-1], -1) * s["scale"]
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(*x.shape[:2], 1, -1, p.shape[-1]), v).view(x.shape)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(*row.shape, heads, dim)
    out = torch.zeros(q.shape, device=DEV)
    out[row[real]] = o[real]
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].float()))
    return out.to(q.dtype)


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------
def _own_kvplan(s):
    import ternary_weight_int8_tb_amd as tb
    tb.tb_kv_plan(s["context"], s["fresh"], s["page"], s["pages"], s["table"], s["free"], s["count"], s["lengths"], s["offsets"], s["positions"],
                  s["slots"], s["left"], s["missing"])
    return {k: s[k] for k in ("table", "free", "left", "lengths", "offsets", "positions", "slots", "missing")}


def _own_rope(s):
    import ternary_weight_int8_tb_amd as tb
    if "handles" not in s:  # the model's frequencies and the cache, made once when a program starts
        layout = tb.TB_ROPE_HALF if s["layout"] == HALF else tb.TB_ROPE_INTERLEAVED
        s["handles"] = tb.Rope(s["freq"], layout, s["factor"]), tb.KvCache(s["kcache"], s["vcache"])
    rope, cache = s["handles"]
    tb.tb_rope_kv(s["q"], s["k"], s["v"], rope, s["positions"], s["slots"], cache, s["out"])
    return {"q": s["out"], "k": s["kcache"], "v": s["vcache"]}


def _own_attn(s):
    import ternary_weight_int8_tb_amd as tb
    if "cache" not in s:
        s["cache"] = tb.KvCache(s["kcache"], s["vcache"])
    tb.tb_attn_paged(s["q"], s["cache"], s["table"], s["offsets"], s["lengths"], s["scale"], s["out"], s["ws"], gate=s["gate"], window=s["window"])
    return s["out"]


def run(state):
    op = state["op"]
    if own:
        return {"kvplan": _own_kvplan, "rope": _own_rope, "attn": _own_attn}[op](state)
    return {"kvplan": _plain_kvplan, "rope": _plain_rope, "attn": _plain_attn}[op](state)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "kvplan":
        page, rows, moved = c["page"], 0, 0
        for context, new in _lengths(c):
            took = min(max(new, 0), c["rows"] - rows)
            rows += took
            pages = -(-context // page)
            # a page given back or taken: an entry of the table and one of the free list
            moved += pages if new < 0 else -(-(context + took) // page) - pages
        return {"bytes": 4 * (4 * c["requests"] + 1 + 2 * c["rows"] + 2 * moved + 3), "flops": 4 * c["rows"]}
    heads, kv, dim = c["heads"], c["kv"], c["dim"]
    if c["op"] == "rope":
        t = c["tokens"] - c["pad"]
        moved = heads * (SIZE[c["rows"]] + SIZE[c["q"]]) + 2 * kv * (SIZE[c["rows"]] + SIZE[c["cache"]])
        return {"bytes": t * dim * moved + 8 * c["tokens"] + 4 * c["rot"], "flops": t * (heads + kv) * c["rot"] * 3}
    rows = keys = seen = 0
    for context, new in _lengths(c):
        first = max(0, context + 1 - c["window"]) if c["window"] else 0
        rows += new
        keys += context + new - first
        # key-query pairs: the i-th new token sees context + i + 1 keys, or the window's
        if c["window"]:
            seen += sum(min(context + i + 1, c["window"]) for i in range(new))
        else:
            seen += new * context + new * (new + 1) // 2
    return {"bytes": keys * kv * dim * 2 * SIZE[c["cache"]] + rows * heads * dim * SIZE[c["rows"]] * (2 + c["gate"]), "flops": 4 * seen * heads * dim}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits (the plan has whole numbers alone)
# ---------------------------------------------------------------------------------------------
def _exact_rope(c, s):
    t, dim, rot = c["tokens"], c["dim"], c["rot"]
    # a pair as a complex number, turned by exp(i * position * frequency)
    turn = torch.polar(torch.full((t, rot // 2), float(s["factor"]), dtype=torch.float64, device=DEV), torch.outer(s["positions"].double(), s["freq"]))
    first = torch.arange(rot // 2, device=DEV) * (1 if c["layout"] == HALF else 2)
    second = first + (rot // 2 if c["layout"] == HALF else 1)
    done = {}
    for name in ("q", "k"):
        x = s[name].double().clone()
        z = torch.complex(x[:, :, first], x[:, :, second]) * turn[:, None, :]
        x[:, :, first], x[:, :, second] = z.real, z.imag
        done[name] = x
    out = done["q"] * (s["positions"] >= 0).double()[:, None, None]
    caches = []
    for rows, like in ((done["k"], s["kcache"]), (s["v"].double(), s["vcache"])):
        flat = torch.zeros(like.shape[0] * c["page"], c["kv"], dim, dtype=torch.float64, device=DEV)
        for first in range(0, t, 4096):
            at = s["slots"][first:first + 4096].long()
            flat[at[at >= 0]] = rows[first:first + 4096][at >= 0]
        caches.append(flat.view(like.shape[0], c["page"], c["kv"], dim).permute(0, 2, 1, 3).contiguous())
    return {"q": out, "k": caches[0], "v": caches[1]}


def _exact_attn(c, s):
    group = c["heads"] // c["kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    start = 0
    for r, (context, new) in enumerate(_lengths(c)):
        n = context + new
        held = s["table"][r, :-(-n // c["page"])].long()
        for h in range(c["kv"]):
            keys = s["kcache"][held, h].reshape(-1, c["dim"])[:n].double()
            values = s["vcache"][held, h].reshape(-1, c["dim"])[:n].double()
            for first in range(0, new, 256):
                last = min(new, first + 256)
                at = torch.arange(context + first, context + last, device=DEV)[:, None]
                j = torch.arange(n, device=DEV)[None]
                hidden = (j > at) | ((j <= at - c["window"]) if c["window"] else False)
                for g in range(h * group, (h + 1) * group):
                    w = s["q"][start + first:start + last, g].double() @ keys.T * s["scale"]
                    w = torch.softmax(w.masked_fill(hidden, -math.inf), 1)
                    out[start + first:start + last, g] = w @ values
        start += new
    return out if s["gate"] is None else out * torch.sigmoid(s["gate"].double())


def exact(case, seed):
    if case["op"] == "kvplan":
        return None
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_attn(case, s)
