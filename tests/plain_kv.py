"""Plain implementations, in whole numbers and 64 bits, of the operators around the paged cache, for the tests. They
share no code with the library."""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24                                  # half a step of fp32, relative
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def plan(context, fresh, rows, page, pages, table, free, count):
    """The step's plan, request by request: a dict of what tb_kv_plan writes. `free`: the whole list, of which `count` count."""
    table, width = table.copy(), table.shape[1]
    stack = [int(x) for x in free[:count]]
    context = [max(int(c), 0) for c in context]
    held = [min(-(-c // page), width) for c in context]
    for s, f in enumerate(fresh):
        if f < 0:
            stack += [int(x) for x in table[s, :held[s]] if 0 <= x < pages]
    offsets, lengths, positions, slots, missing = [0], [], [], [], 0
    news = []
    for s, f in enumerate(fresh):
        n = min(max(int(f), 0), rows - offsets[-1])
        offsets.append(offsets[-1] + n)
        lengths.append(0 if f < 0 else context[s] + n)
        news.append(n)
    for s, f in enumerate(fresh):
        for j in range(held[s], min(-(-lengths[s] // page), width)):
            table[s, j] = stack.pop() if stack else -1
    for s, n in enumerate(news):
        for i in range(n):
            p = lengths[s] - n + i
            entry = int(table[s, p // page]) if p // page < width else -1
            ok = 0 <= entry < pages
            positions.append(p)
            slots.append(entry * page + p % page if ok else -1)
            missing += not ok
    pad = [-1] * (rows - len(positions))
    return {"table": table, "stack": stack, "lengths": lengths, "offsets": offsets, "positions": positions + pad, "slots": slots + pad,
            "left": len(stack), "missing": missing}


def rope(x, positions, freq, factor, interleaved):
    """(rows x [tokens][heads][dim] with the pairs of their first 2 len(freq) elements turned, the sum of each pair's magnitudes)."""
    y = x.astype(np.float64).copy()
    size = np.abs(y)
    n = len(freq)
    angle = positions.astype(np.float64)[:, None] * freq
    c, s = (f(angle)[:, None] * factor for f in (np.cos, np.sin))
    i = np.arange(n)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
    a, b = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    both = (np.abs(a) + np.abs(b)) * factor
    size[..., first] = size[..., second] = both
    return y, size


def attention(q, k, v, table, offsets, lengths, scale, window=0, gate=None):
    """(out, size): the attention of q [tokens][heads][dim] over caches [pages][kv][page][dim], all in 64 bits, and for each element
    the weighted sum of the values' magnitudes; and per row the largest sum of magnitudes in a score, and the number of keys."""
    pages, kv, page, dim = k.shape
    heads = q.shape[1]
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    big, keys = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    for s, n in enumerate(lengths):
        new = offsets[s + 1] - offsets[s]
        for i in range(new):
            p = n - new + i
            lo = max(0, p - window + 1) if window else 0
            js = [j for j in range(lo, min(p + 1, n)) if j // page < table.shape[1] and 0 <= table[s, j // page] < pages]
            if not js:
                continue
            js = np.array(js)
            at, place = table[s, js // page], js % page
            for h in range(heads):
                g = h // (heads // kv)
                kk, vv = k[at, g, place], v[at, g, place]
                x = q[offsets[s] + i, h]
                with np.errstate(all="ignore"):
                    score = (kk @ x) * scale
                    if np.isneginf(score).all():
                        continue
                    w = np.exp(score - score.max())
                    w /= w.sum()
                    out[offsets[s] + i, h] = w @ vv
                    size[offsets[s] + i, h] = w @ np.abs(vv)
                    big[offsets[s] + i, h] = (np.abs(kk) @ np.abs(x)).max() * scale
                    keys[offsets[s] + i, h] = len(js)
    if gate is not None:
        f = 1 / (1 + np.exp(-gate))
        out, size = out * f, size * f
    return out, size, big, keys


def attention_bound(out, size, big, keys, dim, rows, cache):
    """How far a row's elements may be off. To first order, with e the relative error of every weight, o is off by 2 e size
    (numerator and sum):
      - a score: dim products and sums in fp32, 2^-23 of the sum of magnitudes each at most; the factor scale log2(e), its product
        and the maximum's: 4 U of the score; the exponential: 4 U
      - fp32 rows: q's parts keep 22 bits (fp16) or 24: 2^-22 of the score's magnitudes
      - a weight's rounding: half a step of the cache's type, or 2^-22 of fp32 rows' parts
    the sums over the keys: 32 at a time, 2^-23 of size for each such sum, its own and its joining; and for each of the four
    waves and of the parts of a unit, at most 64 of them at the tests' sizes; then the output's type and the gate's 8 U."""
    e = big[..., None] * ((dim + 8) * 2.0 ** -23 + 2.0 ** -22) + 8 * U
    e = e + (2.0 ** -22 if rows == "f32" else HALF_STEP[cache])
    return (2 * e + (keys[..., None] / 16 + 200) * 2.0 ** -23 + 8 * U) * size + HALF_STEP[rows] * np.abs(out) * 1.001 + 1e-37
