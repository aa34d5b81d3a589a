"""Operators around the ternary FFN, each in a plain torch form and as calls of libtb.so.

Four operators, measured on cases of three kinds: the smallest calls (one token, where latency
counts), ordinary ones, and the largest.

  norm      residual addition + root-mean-square norm + rotated int8 rows (what every FFN and
            attention block of the model starts with; its int8 rows are what the ternary and sign
            products read)
  mxquant   rows to microscaled 4-bit floating point (e2m1 elements, one e8m0 scale per 32), with
            or without the 128-block rotation (weights once, activations at every step)
  mxlinear  a layer with microscaled 4-bit weights: quantise the rows, multiply (the layers of a
            ternary model that stay in a 4-bit format: attention projections, head)
  moe       an FFN of ternary or sign experts: sort the (token, expert) pairs, gate/up with SiLU,
            down, and the weighted sum of each token's experts

A case names its operator in "op". Values held in 8 or 4 bits come back as the numbers they stand
for, in bfloat16.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
MXB = 32
UNIT = 1.0 / (127.0 * math.sqrt(128.0))
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TERNARY, SIGN = "ternary", "sign"


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoded token entering an FFN: hidden 5120
        {"name": "norm-1", "op": "norm", "m": 1, "k": 5120, "type": "bf16", "res": True, "y": False},
        # an odd batch at the intermediate width, in fp32, the normed rows wanted too (a router reads them)
        {"name": "norm-37-wide", "op": "norm", "m": 37, "k": 17408, "type": "f32", "res": True, "y": True},
        # a prefill of 8192 tokens
        {"name": "norm-8192", "op": "norm", "m": 8192, "k": 5120, "type": "bf16", "res": True, "y": False},
        # a few decoded tokens' rotated activations
        {"name": "mxquant-rot-5", "op": "mxquant", "m": 5, "k": 5120, "type": "f16", "rotate": True},
        # a whole weight matrix, once at load: 17408 x 5120
        {"name": "mxquant-weights", "op": "mxquant", "m": 17408, "k": 5120, "type": "bf16", "rotate": False},
        # one decoded token through the fused query/gate/key/value projection
        {"name": "mxlinear-1", "op": "mxlinear", "m": 1, "k": 5120, "n": 9216, "type": "bf16", "out": "f32"},
        # 24 concurrent decodes through a down projection
        {"name": "mxlinear-24", "op": "mxlinear", "m": 24, "k": 17408, "n": 5120, "type": "bf16", "out": "bf16"},
        # an odd chunk of a prompt through an output projection
        {"name": "mxlinear-509", "op": "mxlinear", "m": 509, "k": 4096, "n": 5120, "type": "bf16", "out": "bf16"},
        # a long prefill through an up projection
        {"name": "mxlinear-8192", "op": "mxlinear", "m": 8192, "k": 5120, "n": 17408, "type": "bf16", "out": "bf16"},
        # one decoded token, 8 of 64 experts
        {"name": "moe-1", "op": "moe", "tokens": 1, "experts": 64, "topk": 8, "hidden": 2048, "inter": 1024, "fmt": TERNARY, "drop": 0.0},
        # 48 concurrent decodes over wide sign experts, some pairs dropped
        {"name": "moe-48-sign", "op": "moe", "tokens": 48, "experts": 16, "topk": 2, "hidden": 5120, "inter": 2176, "fmt": SIGN, "drop": 0.1},
        # a prefill of 4096 tokens, 8 of 64 experts
        {"name": "moe-4096", "op": "moe", "tokens": 4096, "experts": 64, "topk": 8, "hidden": 2048, "inter": 1024, "fmt": TERNARY, "drop": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "mxquant", "mxlinear", "moe"])
    if op == "norm":
        k = BLOCK * _log(rng, 1, 136)
        return {"op": op, "m": _log(rng, 1, min(8192, 41_943_040 // k)), "k": k, "type": rng.choice(list(TYPES)),
                "res": rng.random() < 0.8, "y": rng.random() < 0.4}
    if op == "mxquant":
        k = BLOCK * _log(rng, 1, 136)
        return {"op": op, "m": _log(rng, 1, min(17408, 89_128_960 // k)), "k": k, "type": rng.choice(list(TYPES)),
                "rotate": rng.random() < 0.5}
    if op == "mxlinear":
        k, n = BLOCK * _log(rng, 1, 136), _log(rng, 16, 17408)
        return {"op": op, "m": _log(rng, 1, min(8192, 730_000_000_000 // (k * n))), "k": k, "n": n,
                "type": rng.choice(list(TYPES)), "out": rng.choice(list(TYPES))}
    experts = rng.choice([2, 4, 8, 16, 32, 64])
    topk = rng.randint(1, min(8, experts))
    hidden, inter = BLOCK * _log(rng, 2, 40), BLOCK * _log(rng, 1, 24)
    while experts * hidden * inter > 134_217_728:
        experts = max(2, experts // 2)
        topk = min(topk, experts)
        inter = max(BLOCK, inter // 2 // BLOCK * BLOCK)
    tokens = _log(rng, 1, min(4096, 68_000_000_000 // (topk * hidden * inter)))
    return {"op": op, "tokens": tokens, "experts": experts, "topk": topk, "hidden": hidden, "inter": inter, "fmt": rng.choice([TERNARY, SIGN]),
            "drop": rng.choice([0.0, 0.0, 0.1, 0.5]) if tokens * topk >= 16 else 0.0}


# ---------------------------------------------------------------------------------------------
# Inputs, and the buffers that a user's program keeps
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def _rows(g, m, k, dtype):
    """Activations: normal, with a few channels ten times as large, as a residual stream has them."""
    x = torch.randn(m, k, generator=g, device=DEV)
    x *= torch.where(torch.rand(k, generator=g, device=DEV) < 0.01, 10.0, 1.0)
    return x.to(dtype)


def _pack(g, fmt, *shape):
    """Random experts: packed codes of shape [..., k/128, 32 or 16] and fp16 scales [..., k/128]."""
    *lead, k = shape
    nb = k // BLOCK
    scales = torch.exp(-4.0 + 0.5 * torch.randn(*lead, nb, generator=g, device=DEV)).to(torch.float16)
    if fmt == SIGN:
        return torch.randint(0, 256, (*lead, nb, 16), generator=g, device=DEV, dtype=torch.uint8), scales
    c = torch.randint(0, 3, (*lead, nb, 32, 4), generator=g, device=DEV, dtype=torch.uint8)
    codes = c[..., 0] | c[..., 1] << 2 | c[..., 2] << 4 | c[..., 3] << 6
    return codes.contiguous(), scales


def _prepare_norm(c, g):
    dt = TYPES[c["type"]]
    m, k = c["m"], c["k"]
    return {"x": _rows(g, m, k, dt), "res": _rows(g, m, k, dt) if c["res"] else None,
            "gamma": 1.0 + 0.2 * torch.randn(k, generator=g, device=DEV),
            "res_out": _empty(m, k, dtype=dt) if c["res"] else None, "y": _empty(m, k, dtype=dt) if c["y"] else None,
            "q": _empty(m, k, dtype=torch.int8), "dq": _empty(m, k // BLOCK), "value": _empty(m, k // BLOCK, BLOCK, dtype=torch.bfloat16)}


def _prepare_mxquant(c, g):
    m, k = c["m"], c["k"]
    return {"x": _rows(g, m, k, TYPES[c["type"]]), "rotate": c["rotate"], "codes": _empty(m, k // 2, dtype=torch.uint8),
            "scales": _empty(m, k // MXB, dtype=torch.uint8), "value": _empty(m, k, dtype=torch.bfloat16)}


def _prepare_mxlinear(c, g):
    m, n, k = c["m"], c["n"], c["k"]
    return {"x": _rows(g, m, k, TYPES[c["type"]]),
            # the codes and scales of a trained layer: every code, scales a few binades around 2^-6
            "w_codes": torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8),
            "w_scales": torch.randint(118, 124, (n, k // MXB), generator=g, device=DEV, dtype=torch.uint8),
            "codes": _empty(m, k // 2, dtype=torch.uint8), "scales": _empty(m, k // MXB, dtype=torch.uint8),
            # scratch that the program keeps for every layer
            "ws": _empty(64 << 20, dtype=torch.uint8), "out": _empty(m, n, dtype=TYPES[c["out"]])}


def _prepare_moe(c, g):
    t, e, topk, hid, inter = c["tokens"], c["experts"], c["topk"], c["hidden"], c["inter"]
    # a router's choice: distinct experts, some more popular than others; a dropped pair has no expert
    logits = torch.randn(t, e, generator=g, device=DEV) + 0.7 * torch.randn(e, generator=g, device=DEV)
    top, ids = torch.topk(logits, topk, dim=1)
    weights = torch.softmax(top, 1)
    ids = torch.where(torch.rand(t, topk, generator=g, device=DEV) < c["drop"], -1, ids).to(torch.int32)
    # rows as the rotating quantiser leaves them: near-normal codes, one scale per block
    u = torch.randn(t, hid // BLOCK, BLOCK, generator=g, device=DEV)
    amax = u.abs().amax(-1, keepdim=True)
    s = {"q": torch.round(u * (127.0 / amax)).to(torch.int8).view(t, hid), "dq": (amax / 127.0).view(t, -1).contiguous(),
         "ids": ids.contiguous(), "weights": weights.contiguous(), "experts": e, "topk": topk, "fmt": c["fmt"],
         "cap": max(1, int(torch.bincount(ids[ids >= 0].long(), minlength=1).max())) if bool((ids >= 0).any()) else 1}
    for name, n, k in (("gate", inter, hid), ("up", inter, hid), ("down", hid, inter)):
        s[name] = _pack(g, c["fmt"], e, n, k)
    p = t * topk
    s |= {"offsets": _empty(e + 1, dtype=torch.int32), "order": _empty(p, dtype=torch.int32), "h": _empty(p, inter),
          "qh": _empty(p, inter, dtype=torch.int8), "dqh": _empty(p, inter // BLOCK), "pairs": _empty(p, hid),
          "out": _empty(t, hid, dtype=torch.bfloat16)}
    return s


_PREPARE = {"norm": _prepare_norm, "mxquant": _prepare_mxquant, "mxlinear": _prepare_mxlinear, "moe": _prepare_moe}


def prepare(case, seed):
    state = _PREPARE[case["op"]](case, _gen(seed))
    state["op"] = case["op"]
    state["H"] = _hadamard()
    return state


def _hadamard():
    """The 128 x 128 Walsh-Hadamard matrix of +1 and -1, by doubling."""
    h = torch.ones(1, 1, device=DEV)
    two = torch.tensor([[1.0, 1.0], [1.0, -1.0]], device=DEV)
    for _ in range(7):
        h = torch.kron(two, h)
    return h


# ---------------------------------------------------------------------------------------------
# Plain forms, in 32 bits
# ---------------------------------------------------------------------------------------------
def _plain_i8(t, H):
    """Rotated rows quantised per 128-block: whole numbers (as fp32) and the blocks' largest magnitude."""
    u = t.reshape(*t.shape[:-1], -1, BLOCK) @ H
    amax = u.abs().amax(-1, keepdim=True)
    q = torch.where(amax > 0, torch.round(u * (127.0 / amax)), 0.0)
    return q, amax


def _plain_norm(s):
    r = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)
    f = r.float()
    inv = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    q, amax = _plain_i8(f * s["gamma"], s["H"])
    dq = amax * (inv[..., None] * UNIT)
    out = {"dq": dq[..., 0], "value": (q * dq).to(torch.bfloat16)}
    if s["res"] is not None:
        out["res"] = r
    if s["y"] is not None:
        out["y"] = (f * inv * s["gamma"]).to(r.dtype)
    return out


def _plain_mx(x, rotate, H):
    """The values that microscaled e2m1 rows stand for, in fp32."""
    f = x.float()
    if rotate:
        f = ((f.view(-1, BLOCK) @ H) * (1.0 / math.sqrt(128.0))).view(f.shape)
    b = f.view(f.shape[0], -1, MXB)
    e = (torch.frexp(b.abs().amax(-1, keepdim=True)).exponent - 3).clamp(-127, 127)
    v = torch.ldexp(b, -e)
    a = v.abs()
    r = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2)).clamp(max=6)
    return torch.ldexp(torch.copysign(r, v), e).view(f.shape)


def _plain_mx_values(codes, scales):
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    v = lut[torch.stack((codes & 15, codes >> 4), -1).int()].view(*scales.shape, MXB)
    return (v * torch.exp2(scales.float() - 127.0)[..., None]).view(scales.shape[0], -1)


def _plain_mxlinear(s):
    y = _plain_mx(s["x"], False, s["H"]) @ _plain_mx_values(s["w_codes"], s["w_scales"]).t()
    return y.to(s["out"].dtype)


def _plain_weights(fmt, packed):
    codes, scales = packed
    if fmt == SIGN:
        t = torch.stack([codes >> i & 1 for i in range(8)], -1).float() * 2 - 1
    else:
        c = torch.stack([codes >> i & 3 for i in range(0, 8, 2)], -1)
        t = (c & 1).float() - (c >> 1).float()
    w = t.view(*scales.shape, BLOCK) * scales.float()[..., None]
    return w.view(*scales.shape[:-1], -1)


def _plain_moe(s):
    e, cap, topk = s["experts"], s["cap"], s["topk"]
    ids = s["ids"].view(-1).long()
    kept = ids >= 0
    gate, up, down = s["gate"], s["up"], s["down"]
    if ids.numel() < e:  # fewer pairs than experts: only the experts that a pair asks for, one row each
        gate, up, down = ((codes[ids.clamp(min=0)], scales[ids.clamp(min=0)]) for codes, scales in (gate, up, down))
        e, cap = ids.numel(), 1
        ids = torch.where(kept, torch.arange(e, device=DEV), -1)
    # each pair's place in its expert's padded list (a dropped pair goes to a row of its own behind them)
    hot = torch.nn.functional.one_hot(torch.where(kept, ids, e), e + 1)
    place = (hot.cumsum(0) - 1).gather(1, torch.where(kept, ids, e)[:, None])[:, 0]
    slot = torch.where(kept, ids * cap + place, e * cap)
    a = s["q"].float().view(*s["dq"].shape, BLOCK) * s["dq"][..., None]
    a = a.view(s["q"].shape[0], -1).repeat_interleave(topk, 0)
    x = torch.zeros(e * cap + 1, a.shape[1], device=DEV)
    x[slot] = a
    x = x[:-1].view(e, cap, -1)
    g = x @ _plain_weights(s["fmt"], gate).transpose(1, 2)
    u = x @ _plain_weights(s["fmt"], up).transpose(1, 2)
    h = g / (1 + torch.exp(-g)) * u
    q, amax = _plain_i8(h, s["H"])
    y = (q * (amax * UNIT)).view(h.shape) @ _plain_weights(s["fmt"], down).transpose(1, 2)
    y = torch.cat((y.reshape(e * cap, -1), torch.zeros(1, y.shape[-1], device=DEV)))
    out = (y[slot].view(-1, topk, y.shape[-1]) * s["weights"][..., None]).sum(1)
    return out.to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------
def _own_norm(s):
    import ternary_weight_int8_tb_amd as tb
    tb.tb_add_rmsnorm_quant_i8(s["x"], s["res"], s["gamma"], EPS, s["res_out"], s["y"], s["q"], s["dq"])
    torch.mul(s["q"].view(s["value"].shape), s["dq"][..., None], out=s["value"])
    out = {"dq": s["dq"], "value": s["value"]}
    if s["res"] is not None:
        out["res"] = s["res_out"]
    if s["y"] is not None:
        out["y"] = s["y"]
    return out


def _own_mxquant(s):
    import ternary_weight_int8_tb_amd as tb
    tb.tb_mxfp4_quant(s["x"], s["codes"], s["scales"], rotate=s["rotate"])
    tb.tb_mxfp4_dequant(s["codes"], s["scales"], s["value"])
    return s["value"]


def _own_mxlinear(s):
    import ternary_weight_int8_tb_amd as tb
    if "layer" not in s:  # the layer's handle, made once when a program loads its weights
        s["layer"] = tb.Mxfp4(s["w_codes"], s["w_scales"])
    tb.tb_mxfp4_quant(s["x"], s["codes"], s["scales"])
    tb.tb_mxfp4_gemm(s["layer"], s["codes"], s["scales"], s["out"], s["ws"])
    return s["out"]


def _own_moe(s):
    import ternary_weight_int8_tb_amd as tb
    if "layer" not in s:
        fmt = tb.TB_FMT_SIGN1 if s["fmt"] == SIGN else tb.TB_FMT_TERNARY2
        s["layer"] = [tb.Experts(*s[n], fmt) for n in ("gate", "up", "down")]
    gate, up, down = s["layer"]
    tb.tb_moe_plan(s["ids"], s["experts"], s["offsets"], s["order"])
    tb.tb_moe_gateup_silu(gate, up, s["q"], s["dq"], s["topk"], s["offsets"], s["order"], s["h"], s["qh"], s["dqh"])
    tb.tb_moe_down(down, s["qh"], s["dqh"], s["offsets"], s["order"], s["pairs"])
    tb.tb_moe_combine(s["pairs"], s["weights"], s["ids"], s["experts"], s["out"])
    return s["out"]


def run(state):
    op = state["op"]
    if own:
        return {"norm": _own_norm, "mxquant": _own_mxquant, "mxlinear": _own_mxlinear, "moe": _own_moe}[op](state)
    if op == "norm":
        return _plain_norm(state)
    if op == "mxquant":
        return _plain_mx(state["x"], state["rotate"], state["H"]).to(torch.bfloat16)
    return _plain_mxlinear(state) if op == "mxlinear" else _plain_moe(state)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if c["op"] == "norm":
        m, k, b = c["m"], c["k"], size[c["type"]]
        io = b * (1 + 2 * c["res"] + c["y"]) + 1
        return {"bytes": m * k * io + m * k // BLOCK * 4 + 4 * k, "flops": m * k * (7 + 8)}
    if c["op"] == "mxquant":
        m, k = c["m"], c["k"]
        return {"bytes": m * k * size[c["type"]] + m * k // 2 + m * k // MXB, "flops": m * k * (4 + 8 * c["rotate"])}
    if c["op"] == "mxlinear":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": m * k * size[c["type"]] + n * k // 2 + n * k // MXB + m * n * size[c["out"]], "flops": 2 * m * n * k}
    t, hid, inter = c["tokens"], c["hidden"], c["inter"]
    pairs = t * c["topk"] * (1 - c["drop"])
    # experts that get a pair, were the router even
    used = c["experts"] * (1 - (1 - 1 / c["experts"]) ** pairs)
    block = (32 if c["fmt"] == TERNARY else 16) + 2
    return {"bytes": int(used * 3 * hid * inter // BLOCK * block) + t * hid * 3, "flops": int(2 * pairs * 3 * hid * inter)}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _signs64():
    """H[i][j] = (-1)^popcount(i & j), by counting bits."""
    i = torch.arange(BLOCK, device=DEV)
    both = i[:, None] & i[None, :]
    ones = sum((both >> b) & 1 for b in range(7))
    return 1.0 - 2.0 * (ones % 2).double()


def _exact_i8(rows):
    """(whole numbers, scale of one step) of rotated rows, 128 at a time."""
    u = torch.einsum("rbj,ij->rbi", rows.reshape(rows.shape[0], -1, BLOCK), _signs64())
    big = u.abs().max(-1, keepdim=True).values
    step = big / 127
    return torch.where(big > 0, (u / torch.where(big > 0, step, 1.0)).round(), 0.0), step / math.sqrt(BLOCK)


def _exact_norm(c, s):
    total = s["x"].double() + (s["res"].double() if c["res"] else 0.0)
    kept = total.to(TYPES[c["type"]]).double()  # the residual is what was stored
    rms = torch.sqrt((kept * kept).sum(1, keepdim=True) / c["k"] + EPS)
    q, step = _exact_i8(kept * s["gamma"].double())
    step = step / rms[..., None]
    out = {"dq": step[..., 0], "value": q * step}
    if c["res"]:
        out["res"] = kept
    if c["y"]:
        out["y"] = kept / rms * s["gamma"].double()
    return out


def _exact_mx(x, rotate):
    f = x.double()
    if rotate:
        f = torch.einsum("rj,ij->ri", f.reshape(-1, BLOCK), _signs64()).reshape(f.shape) / math.sqrt(BLOCK)
    f = f.reshape(f.shape[0], -1, MXB)
    big = f.abs().max(-1, keepdim=True).values
    scale = torch.where(big > 0, torch.exp2(torch.floor(torch.log2(torch.where(big > 0, big, 1.0))) - 2), 1.0)
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    middle = (levels[1:] + levels[:-1]) / 2
    a = (f.abs() / scale).contiguous()
    # the number of borders below: a tie goes to the level with an even index
    below, upto = torch.searchsorted(middle, a), torch.searchsorted(middle, a, right=True)
    index = torch.where(below == upto, below, torch.where(below % 2 == 0, below, upto))
    return (levels[index] * scale * torch.where(f < 0, -1.0, 1.0)).reshape(x.shape)


def _exact_mxlinear(c, s):
    codes, n, k = s["w_codes"].int(), c["n"], c["k"]
    e2m1 = torch.stack((codes % 16, codes // 16), 2).reshape(n, k)
    mag = e2m1 % 8
    exponent, mantissa = mag // 2, (mag % 2).double()
    w = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * torch.exp2((exponent - 1).double()))
    w = w * (1 - 2 * (e2m1 // 8).double())
    w = w.reshape(n, -1, MXB) * torch.exp2(s["w_scales"].double() - 127)[..., None]
    return _exact_mx(s["x"], False) @ w.reshape(n, k).T


def _exact_expert(fmt, packed, e):
    codes, scales = packed[0][e].long(), packed[1][e].double()
    if fmt == SIGN:
        t = ((codes[..., None] // (2 ** torch.arange(8, device=DEV))) % 2) * 2 - 1
    else:
        t = torch.tensor([0, 1, -1, 0], device=DEV)[(codes[..., None] // (4 ** torch.arange(4, device=DEV))) % 4]
    return (t.reshape(*scales.shape, BLOCK) * scales[..., None]).reshape(scales.shape[0], -1)


def _exact_moe(c, s):
    x = (s["q"].double().reshape(*s["dq"].shape, BLOCK) * s["dq"].double()[..., None]).reshape(c["tokens"], -1)
    out = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device=DEV)
    for e in range(c["experts"]):
        token, j = (s["ids"] == e).nonzero(as_tuple=True)
        if len(token):
            gate, up, down = (_exact_expert(c["fmt"], s[n], e) for n in ("gate", "up", "down"))
            g, u = x[token] @ gate.T, x[token] @ up.T
            q, step = _exact_i8(g * torch.sigmoid(g) * u)
            y = (q * step).reshape(len(token), -1) @ down.T
            out.index_add_(0, token, y * s["weights"][token, j].double()[:, None])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "mxquant":
        return _exact_mx(s["x"], case["rotate"])
    return _exact_mxlinear(case, s) if case["op"] == "mxlinear" else _exact_moe(case, s)
