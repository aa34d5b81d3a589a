"""Block tables and slots of a step, and rotary positions into the paged cache, on MI355X, against plain implementations."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import ternary_weight_int8_tb_amd as tb
from tests import gpu_util as gu
from tests import plain_kv
from tests.plain_kv import HALF_STEP, U

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield


def ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device=gu.DEV)


class Step:
    """Buffers of a plan, the outputs poisoned."""

    def __init__(self, context, fresh, rows, page, pages, table, free, count, in_place=False):
        n = len(context)
        self.page, self.pages = page, pages
        self.context, self.fresh, self.table, self.free, self.count = (ints(x) for x in (context, fresh, table, free, [count]))
        self.lengths = self.context if in_place else gu.i32_out(n)
        self.left = self.count if in_place else gu.i32_out(1)
        self.offsets, self.positions, self.slots, self.missing = gu.i32_out(n + 1), gu.i32_out(rows), gu.i32_out(rows), gu.i32_out(1)

    def run(self, stream=None):
        tb.tb_kv_plan(self.context, self.fresh, self.page, self.pages, self.table, self.free, self.count, self.lengths, self.offsets,
                      self.positions, self.slots, self.left, self.missing, stream)

    def check(self, want):
        left = int(gu.host(self.left)[0])
        assert left == want["left"] and int(gu.host(self.missing)[0]) == want["missing"]
        for name in ("lengths", "offsets", "positions", "slots"):
            assert gu.host(getattr(self, name)).tolist() == want[name], name
        assert np.array_equal(gu.host(self.table), want["table"])
        assert gu.host(self.free)[:left].tolist() == want["stack"]


def some_step(rng, n, page, rows, most_context, most_new, spare, width=None, kinds=(0.7, 0.15, 0.1)):
    """Requests of random lengths with pages in random order: arguments of plain_kv.plan."""
    context = rng.integers(0, most_context + 1, n)
    kind = rng.random(n)
    a, b, c = np.cumsum(kinds)
    fresh = np.where(kind < a, 1, np.where(kind < b, rng.integers(0, most_new + 1, n), np.where(kind < c, -1, 0)))
    width = width or max(1, -(-(most_context + most_new) // page))
    held = np.minimum(-(-context // page), width)
    pages = int(held.sum()) + spare
    ids = rng.permutation(pages)
    table = np.full((n, width), -1)
    at = 0
    for s, h in enumerate(held):
        table[s, :h] = ids[at:at + h]
        at += h
    free = np.full(pages, -1)
    free[:spare] = ids[at:]
    return context, fresh, rows, page, pages, table, free, spare


@pytest.mark.parametrize("n,page,rows,most_context,most_new,spare", [
    (1, 16, 1, 0, 1, 1), (1, 16, 5, 40, 9, 4), (3, 32, 7, 70, 2, 3), (17, 16, 300, 100, 60, 80), (64, 256, 64, 3000, 1, 64),
    (255, 16, 2049, 500, 300, 3000), (1025, 64, 1100, 900, 40, 2000), (3000, 16, 9001, 200, 33, 5000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(n, page, rows, most_context, most_new, spare, in_place):
    print(f"kv plan n={n} page={page} rows={rows} in_place={in_place}", flush=True)
    args = some_step(np.random.default_rng(n * page), n, page, rows, most_context, most_new, spare)
    step = Step(*args, in_place=in_place)
    step.run()
    step.check(plain_kv.plan(*args))


def test_plan_without_pages_rows_or_width():
    """Pages run out, rows run out, positions lie beyond the table."""
    rng = np.random.default_rng(3)
    for spare, rows, width in ((0, 40, None), (2, 40, None), (50, 3, None), (50, 200, 2), (1, 1, 1)):
        args = some_step(rng, 9, 16, rows, 60, 20, spare, width, kinds=(0.3, 0.6, 0.1))
        step = Step(*args)
        step.run()
        want = plain_kv.plan(*args)
        step.check(want)


def test_plan_strange_entries():
    """Table rows of ended requests hold entries that name no page, and so does the free list; negative contexts."""
    rng = np.random.default_rng(4)
    context, fresh, rows, page, pages, table, free, count = some_step(rng, 40, 16, 200, 300, 30, 60, kinds=(0.3, 0.3, 0.4))
    hit = rng.random(table.shape) < 0.2
    table = np.where(hit, rng.choice([-1, -7, pages, 2 ** 31 - 1, -2 ** 31], table.shape), table)
    free[:count] = np.where(rng.random(count) < 0.2, pages + 3, free[:count])
    context[5] = -4
    args = (context, fresh, rows, page, pages, table, free, count)
    step = Step(*args)
    step.run()
    step.check(plain_kv.plan(*args))


def test_plan_all_end_or_wait():
    for f in (-1, 0):
        args = list(some_step(np.random.default_rng(5), 70, 32, 9, 400, 1, 5))
        args[1] = np.full(70, f)
        step = Step(*args)
        step.run()
        step.check(plain_kv.plan(*args))


def test_plan_one_long_prompt():
    args = list(some_step(np.random.default_rng(6), 2, 16, 20000, 50000, 20000, 1300, kinds=(0.0, 1.0, 0.0)))
    args[1] = np.array([0, 20000])
    step = Step(*args)
    step.run()
    step.check(plain_kv.plan(*args))


def test_plan_in_a_graph():
    """A captured plan, in place, replayed as requests grow, with other work between the replays."""
    rng = np.random.default_rng(7)
    args = some_step(rng, 30, 16, 64, 100, 1, 400, width=16, kinds=(1.0, 0.0, 0.0))
    step = Step(*args, in_place=True)
    step.run()
    torch.cuda.synchronize()
    want = plain_kv.plan(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for turn in range(5):
        fresh = np.where(rng.random(30) < 0.1, -1, rng.integers(0, 3, 30))
        step.fresh.copy_(ints(fresh))
        free = np.full(args[4], -1)
        free[:want["left"]] = want["stack"]
        want = plain_kv.plan(want["lengths"], fresh, 64, 16, args[4], want["table"], free, want["left"])
        graph.replay()
        step.check(want)
        torch.randn(1000, device=gu.DEV).sum().item()


def test_plan_refusals():
    args = some_step(np.random.default_rng(8), 4, 16, 8, 40, 4, 9)
    for name, bad in (("fresh", torch.zeros(5, dtype=I32, device=gu.DEV)), ("context", torch.zeros(4, dtype=torch.int64, device=gu.DEV)),
                      ("table", torch.zeros(4, 8, dtype=I32, device=gu.DEV)[:, ::2]), ("offsets", torch.zeros(4, dtype=I32, device=gu.DEV)),
                      ("slots", torch.zeros(9, dtype=I32, device=gu.DEV)), ("positions", torch.zeros(8, 1, dtype=I32, device=gu.DEV)),
                      ("count", torch.zeros(1, dtype=I32)), ("free", torch.zeros(1, dtype=I32, device=gu.DEV))):
        step = Step(*args)
        setattr(step, name, bad)
        with pytest.raises(tb.TbError) as e:
            step.run()
        assert e.value.status == tb.TB_EINVAL, name
    step = Step(*args)
    step.page = 24
    with pytest.raises(tb.TbError):
        step.run()


# ---- rotary positions --------------------------------------------------------------------
def rope_case(t, heads, kv, dim, rot, rows, gate=True, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + t * 7 + dim)
    wide = heads * dim * (2 if gate else 1)
    fused = (torch.randn(t, wide + 2 * kv * dim, generator=g) * scale).to(TYPES[rows]).to(gu.DEV)
    view = (lambda at, n: fused[:, at:at + n * dim].view(t, n, dim))
    return view(0, heads), view(wide, kv), view(wide + kv * dim, kv)


def check_rope(got, x, positions, freq, factor, interleaved, dtype):
    want, size = plain_kv.rope(x, positions, freq, factor, interleaved)
    # cos and sin: 2 ulp of the function, the angle's rounding (2^-24 of at most pi / 4), the factor's product, and the angle's own in
    # fp64 (2^-51 of it); then two products and a sum in fp32, and the output's type
    far = (np.abs(positions).max() * np.abs(freq).max()) * 2.0 ** -51
    bound = size * (8 * U + far) + HALF_STEP[dtype] * np.abs(want) * 1.0001 + (6e-8 if dtype == "f16" else 1e-37)
    assert np.all(np.abs(got - want) <= bound), (np.abs(got - want) / bound).max()


@pytest.mark.parametrize("t,heads,kv,dim,rot,page", [(1, 16, 2, 256, 64, 16), (3, 16, 2, 256, 256, 64), (37, 24, 8, 128, 128, 32), (5, 3, 1, 64, 32, 16),
                                                     (70, 5, 5, 96, 48, 128), (2, 1, 1, 16, 16, 16), (9, 7, 2, 512, 368, 256), (130, 8, 2, 80, 16, 16)])
@pytest.mark.parametrize("rows,out,cached", [("f32", "f32", "bf16"), ("f32", "bf16", "bf16"), ("f32", "f16", "f16"), ("bf16", "bf16", "bf16"),
                                             ("f16", "f16", "f16"), ("bf16", "f32", "f16")])
@pytest.mark.parametrize("layout", [tb.TB_ROPE_HALF, tb.TB_ROPE_INTERLEAVED])
def test_rope(t, heads, kv, dim, rot, page, rows, out, cached, layout):
    print(f"rope t={t} heads={heads}/{kv} dim={dim} rot={rot} {rows} {out} {cached} layout={layout}", flush=True)
    rng = np.random.default_rng(t + dim)
    q, k, v = rope_case(t, heads, kv, dim, rot, rows)
    freq, factor = tb.Rope.frequencies(rot, 10000.0, "parts", 4.0, trained=4096)
    rope = tb.Rope(freq.to(gu.DEV), layout, factor)
    positions = rng.integers(0, 1000000, t)
    positions[0] = 0
    pages = t // page + 3
    slots = rng.permutation(pages * page)[:t]
    if t > 4:
        positions[2], slots[2] = -1, -1        # padding
        positions[3] = -5
        slots[4] = pages * page                # no slot: q alone
        slots[1] = -1
    kc = torch.full((pages, kv, page, dim), 7.0, dtype=TYPES[cached], device=gu.DEV)
    vc = torch.full_like(kc, 9.0)
    y = torch.full((t, heads, dim), 5.0, dtype=TYPES[out], device=gu.DEV)
    tb.tb_rope_kv(q, k, v, rope, ints(positions), ints(slots), tb.KvCache(kc, vc), y)
    real = positions >= 0
    got = y.float().cpu().numpy()
    assert np.all(got[~real] == 5.0)
    f64 = freq.numpy()
    ff = float(np.float32(factor))
    inter = layout == tb.TB_ROPE_INTERLEAVED
    check_rope(got[real], q.float().cpu().numpy()[real], positions[real], f64, ff, inter, out)
    kept = real & (slots >= 0) & (slots < pages * page)
    gk, gv = (x.float().cpu().numpy() for x in (kc, vc))
    at, place = slots[kept] // page, slots[kept] % page
    check_rope(gk[at, :, place], k.float().cpu().numpy()[kept], positions[kept], f64, ff, inter, cached)
    assert np.array_equal(gv[at, :, place], v.to(TYPES[cached]).float().cpu().numpy()[kept])
    gk[at, :, place], gv[at, :, place] = 7.0, 9.0
    assert np.all(gk == 7.0) and np.all(gv == 9.0)      # nothing beside the slots


def test_rope_far_positions():
    """The last positions that an int holds, against the angle in long double."""
    t, heads, dim, rot = 8, 2, 64, 64
    q, _, _ = rope_case(t, heads, 1, dim, rot, "f32")
    freq, _ = tb.Rope.frequencies(rot)
    positions = np.array([2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30, 16777217, 10 ** 9, 123456789, 1, 0])
    y = torch.empty(t, heads, dim, device=gu.DEV)
    tb.tb_rope_kv(q, None, None, tb.Rope(freq.to(gu.DEV)), ints(positions), None, None, y)
    x = q.cpu().numpy()
    angle = positions.astype(np.longdouble)[:, None] * freq.numpy().astype(np.longdouble)
    want, size = plain_kv.rope(x, np.ones(t), np.zeros(rot // 2), 1.0, False)
    c, s = np.cos(angle)[:, None].astype(np.float64), np.sin(angle)[:, None].astype(np.float64)
    want[..., :32], want[..., 32:] = x[..., :32] * c - x[..., 32:] * s, x[..., 32:] * c + x[..., :32] * s
    # fp64: the product and its scaling to quarter turns, half a step each; the constant 2/pi, one more; sums
    bound = size * (8 * U + (positions[:, None, None].astype(np.float64)) * 2.0 ** -51) + U * np.abs(want)
    assert np.all(np.abs(y.cpu().numpy() - want) <= bound)


def test_rope_parts_of_the_call():
    """Without a rotation, q alone, and keys and values alone; broadcast rows."""
    t, heads, kv, dim, page = 11, 4, 2, 128, 16
    q, k, v = rope_case(t, heads, kv, dim, dim, "bf16")
    positions, slots = ints(np.arange(t)), ints(np.arange(t) + 3)
    cache = tb.KvCache(*(torch.zeros(2, kv, page, dim, dtype=torch.bfloat16, device=gu.DEV) for _ in range(2)))
    y = torch.zeros(t, heads, dim, dtype=torch.bfloat16, device=gu.DEV)
    tb.tb_rope_kv(q, k, v, None, positions, slots, cache, y)
    assert torch.equal(y, q)
    flat = cache.k.transpose(1, 2).reshape(-1, kv, dim)
    assert torch.equal(flat[3:3 + t], k) and not flat[:3].any() and not flat[3 + t:].any()
    rope = tb.Rope.make(64)
    full = torch.zeros_like(y)
    both = tb.KvCache(torch.zeros_like(cache.k), torch.zeros_like(cache.v))
    tb.tb_rope_kv(q, k, v, rope, positions, slots, both, full)
    alone = torch.zeros_like(y)
    tb.tb_rope_kv(q, None, None, rope, positions, None, None, alone)
    only = tb.KvCache(torch.zeros_like(cache.k), torch.zeros_like(cache.v))
    tb.tb_rope_kv(None, k, v, rope, positions, slots, only, None)
    assert torch.equal(full, alone) and torch.equal(both.k, only.k) and torch.equal(both.v, only.v)
    one = q[:1].expand(t, heads, dim)      # row stride 0
    tb.tb_rope_kv(one, None, None, rope, positions, None, None, alone)
    tb.tb_rope_kv(one.contiguous(), None, None, rope, positions, None, None, full)
    assert torch.equal(alone, full)


def test_rope_past_4_gib():
    """Rows and slots whose places 32 bits cannot count."""
    kv, dim, page, pages = 8, 256, 256, 4200          # 4200 * 8 * 256 * 256 * 2 bytes
    cache = tb.KvCache(torch.zeros(pages, kv, page, dim, dtype=torch.bfloat16, device=gu.DEV),
                       torch.zeros(pages, kv, page, dim, dtype=torch.bfloat16, device=gu.DEV))
    t = 3
    wide = torch.zeros(t, 1 << 30, dtype=torch.bfloat16, device=gu.DEV)     # rows 2 GiB apart
    k = wide[:, :kv * dim].view(t, kv, dim)
    k.copy_(torch.randn(t, kv, dim, device=gu.DEV))
    slots = [pages * page - 1, pages * page - 300, 5]
    rope = tb.Rope.make(128)
    tb.tb_rope_kv(None, k, k, rope, ints([7, 8, 9]), ints(slots), cache, None)
    for i, s in enumerate(slots):
        assert torch.equal(cache.v[s // page, :, s % page], k[i])
        want, _ = plain_kv.rope(k[i:i + 1].float().cpu().numpy(), np.array([7 + i]), rope.freq.cpu().numpy(), 1.0, False)
        assert np.abs(cache.k[s // page, :, s % page].float().cpu().numpy() - want[0]).max() < 0.04
    assert int(torch.count_nonzero(cache.v.sum(-1, dtype=torch.float32))) <= t * kv


def test_rope_refusals():
    t, heads, kv, dim, page = 4, 4, 2, 64, 16
    q, k, v = rope_case(t, heads, kv, dim, dim, "bf16")
    p = ints(np.arange(t))
    cache = tb.KvCache(*(torch.zeros(2, kv, page, dim, dtype=torch.bfloat16, device=gu.DEV) for _ in range(2)))
    y = torch.zeros(t, heads, dim, dtype=torch.bfloat16, device=gu.DEV)
    rope = tb.Rope.make(64)
    good = dict(q=q, k=k, v=v, rope=rope, positions=p, slots=p, cache=cache, q_out=y)
    wide = torch.zeros(t, heads, 2 * dim, dtype=torch.bfloat16, device=gu.DEV)
    for bad in (dict(q=None), dict(q_out=None), dict(k=None), dict(slots=None), dict(q=q.cpu()), dict(q=wide[..., ::2]), dict(k=k[:3]), dict(v=v.float()),
                dict(positions=p.long()), dict(slots=p[:3]), dict(q_out=y[:, :2]), dict(k=torch.cat([k, k], 1)), dict(rope=tb.Rope.make(128)),
                dict(q=q.float()), dict(q_out=y.double())):
        with pytest.raises(tb.TbError) as e:
            tb.tb_rope_kv(**{**good, **bad})
        assert e.value.status == tb.TB_EINVAL, bad.keys()
    with pytest.raises(tb.TbError) as e:      # rows that begin off 16 bytes
        tb.tb_rope_kv(**{**good, "q": torch.zeros(t, heads * dim + 8, dtype=torch.bfloat16, device=gu.DEV)[:, 4:-4].view(t, heads, dim)})
    assert e.value.status == tb.TB_EALIGN
    for bad in (torch.zeros(2, kv, page, dim, device=gu.DEV), torch.zeros(2, kv, dim, dtype=torch.bfloat16, device=gu.DEV)):
        with pytest.raises(tb.TbError):
            tb.KvCache(bad, bad)
    with pytest.raises(tb.TbError):
        tb.Rope(torch.zeros(32, device=gu.DEV))
