"""Attention over a paged cache on MI355X, against a plain implementation in 64 bits."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import ternary_weight_int8_tb_amd as tb
from tests import gpu_util as gu
from tests import plain_kv

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
KINDS = [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield


def ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device=gu.DEV)


class Case:
    """Requests of (length, new tokens) over pages in random order; slots that no request uses hold NaN."""

    def __init__(self, requests, heads, kv, dim, page, rows, cache, seed=0, spread=1.0, spare_width=1, pages=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv, self.dim, self.page, self.rows, self.cached = heads, kv, dim, page, rows, cache
        self.lengths = [n for n, _ in requests]
        self.offsets = np.cumsum([0] + [m for _, m in requests])
        self.tokens = int(self.offsets[-1])
        held = [-(-n // page) for n in self.lengths]
        self.pages = pages or sum(held) + 2
        ids = rng.permutation(self.pages)
        self.table = np.full((len(requests), max(held) + spare_width), -1, np.int32)
        self.k = torch.full((self.pages, kv, page, dim), float("nan"))
        self.v = torch.full((self.pages, kv, page, dim), float("nan"))
        at = 0
        for s, h in enumerate(held):
            self.table[s, :h] = ids[at:at + h]
            at += h
            for j, p in enumerate(self.table[s, :h]):
                n = min(page, self.lengths[s] - j * page)
                self.k[p, :, :n] = torch.randn(kv, n, dim, generator=g) * spread
                self.v[p, :, :n] = torch.randn(kv, n, dim, generator=g) + 0.5
        self.k, self.v = (x.to(TYPES[cache]) for x in (self.k, self.v))
        self.q = torch.randn(self.tokens, heads, dim, generator=g).to(TYPES[rows])
        self.gate, self.window, self.scale = None, 0, float(np.float32(dim ** -0.5))

    def set(self, s, position, k=None, v=None):
        """The key or value of a request's position in every head."""
        p, i = self.table[s, position // self.page], position % self.page
        if k is not None:
            self.k[p, :, i] = k
        if v is not None:
            self.v[p, :, i] = v

    def upload(self, extra=0):
        self.dq, self.dk, self.dv = (x.to(gu.DEV) for x in (self.q, self.k, self.v))
        self.handle = tb.KvCache(self.dk, self.dv)
        self.dt, self.do, self.dl = ints(self.table), ints(self.offsets), ints(self.lengths)
        self.out = torch.full((self.tokens + extra, self.heads, self.dim), 77.0, dtype=self.q.dtype, device=gu.DEV)
        if extra:
            self.dq = torch.cat([self.dq, torch.full((extra, self.heads, self.dim), float("nan"), dtype=self.q.dtype, device=gu.DEV)])
        need = tb.tb_attn_paged_workspace_bytes(self.handle, self.heads, self.q.dtype, len(self.lengths), self.tokens + extra)
        self.ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=gu.DEV)     # NaN, whatever is read of it unwritten
        self.dg = None if self.gate is None else self.gate.to(gu.DEV)
        return self

    def run(self, stream=None):
        tb.tb_attn_paged(self.dq, self.handle, self.dt, self.do, self.dl, self.scale, self.out, self.ws, gate=self.dg, window=self.window,
                         stream=stream)
        return self

    def want(self):
        gate = None if self.gate is None else self.gate.double().numpy()
        return plain_kv.attention(self.q.double().numpy(), self.k.double().numpy(), self.v.double().numpy(), self.table, self.offsets, self.lengths,
                                  self.scale, self.window, gate)

    def check(self, want=None):
        torch.cuda.synchronize()
        got = self.out[:self.tokens].double().cpu().numpy()
        out, size, big, keys = self.want() if want is None else want
        bound = plain_kv.attention_bound(out, size, big, keys, self.dim, self.rows, self.cached)
        if self.rows == "f16":
            bound = bound + 6e-8
        fine = np.isfinite(out)
        assert np.array_equal(fine, np.isfinite(got)) and np.isnan(got[np.isnan(out)]).all()
        if self.rows != "f32":
            # Of fp32 rows a weight has two or three parts, some of them zero (of 0.5 all but the first are): zero times an infinite
            # value is NaN, so that where the formula has an infinity the parts' sum may have NaN. One part is never zero here.
            inf = np.isinf(out)
            assert np.array_equal(out[inf], got[inf])
        off = np.abs(got - out)[fine] / bound[fine]
        assert off.size == 0 or off.max() <= 1, (float(off.max()), np.argwhere(fine)[off.argmax()])
        return float(off.max()) if off.size else 0.0


def say(*a):
    print(*a, flush=True)


@pytest.mark.parametrize("rows,cache", KINDS)
@pytest.mark.parametrize("heads,kv,dim,page", [(16, 2, 256, 16), (6, 2, 128, 32), (5, 1, 64, 64), (3, 3, 64, 16)])
@pytest.mark.parametrize("requests", [[(1, 1)], [(17, 1)], [(33, 33)], [(5, 2), (300, 1), (0, 0), (64, 64), (129, 7)], [(700, 1)], [(257, 40), (16, 16)]])
def test_attention(heads, kv, dim, page, rows, cache, requests):
    say(f"attention {heads}/{kv} dim={dim} page={page} {rows}/{cache} {requests}")
    Case(requests, heads, kv, dim, page, rows, cache, seed=dim + page).upload().run().check()


@pytest.mark.parametrize("rows,cache", KINDS)
@pytest.mark.parametrize("window", [1, 5, 16, 100, 10000, 2 ** 31 - 1])
def test_window(rows, cache, window):
    say(f"window {window} {rows}/{cache}")
    c = Case([(300, 1), (90, 90), (40, 3), (257, 70)], 4, 2, 128, 16, rows, cache, seed=window % 97)
    c.window = window
    c.upload().run().check()


@pytest.mark.parametrize("rows,cache", KINDS)
def test_long_and_split(rows, cache):
    """A unit's keys over many workgroups; beside it short ones; scores that grow along the keys."""
    c = Case([(6000, 1), (3, 1), (2500, 5)], 8, 2, 256, 64, rows, cache, seed=3, spread=2.0)
    for j in range(0, 6000, 500):
        c.set(0, j, k=c.q[0, 0].double() * (j / 6000) / 2)
    c.upload().run().check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("gate", ["f32", "bf16", "f16"])
def test_gate_and_strides(dim, gate):
    """q and the gate as views of wider rows, gates of any type, of any magnitude."""
    c = Case([(40, 9), (130, 2)], 6, 2, dim, 16, "bf16", "bf16", seed=dim)
    wide = torch.randn(c.tokens, 3 * 6 * dim + 64, dtype=torch.float32).to(TYPES[gate])
    wide[0, 6 * dim:6 * dim + 8] = torch.tensor([0.0, 100.0, -100.0, 30.0, -30.0, 1e4, -1e4, -0.0])
    c.gate = wide[:, 6 * dim:12 * dim].view(c.tokens, 6, dim)
    c.upload()
    rows = torch.full((c.tokens, 6 * 2 * dim), float("nan"), dtype=torch.bfloat16, device=gu.DEV)
    view = rows.view(c.tokens, 6, 2 * dim)[:, :, dim:]          # heads interleaved with others
    view.copy_(c.dq)
    c.dq = view
    c.dg = wide.to(gu.DEV)[:, 6 * dim:12 * dim].view(c.tokens, 6, dim)
    c.run().check()


def test_rows_that_see_nothing():
    """More new tokens than the length has (positions below 0), and no length at all: zeros. Rows of no request stay."""
    for rows, cache in KINDS:
        c = Case([(4, 4), (20, 6)], 4, 2, 64, 16, rows, cache, seed=1)
        c.upload(extra=5)
        c.lengths = [2, 0]
        c.dl = ints(c.lengths)
        c.run().check()
        got = c.out.float().cpu().numpy()
        assert not got[:2].any() and not got[4:10].any() and got[2:4].all() and np.all(got[10:] == 77.0)


def test_pages_that_are_none():
    """Entries of the table outside the cache: their keys are left out; a request with none has zeros; so with lengths past the table."""
    for rows, cache in KINDS:
        c = Case([(200, 3), (90, 2), (40, 1)], 4, 2, 128, 16, rows, cache, seed=2)
        c.table[0, 1], c.table[0, 5], c.table[0, 12] = -1, c.pages, 2 ** 31 - 1
        c.table[1] = -5
        c.upload().run().check()
        assert not c.out[3:5].any()
        c.table = np.ascontiguousarray(c.table[:, :4])          # 64 tokens wide: the rest is left out
        c.upload().run().check()


@pytest.mark.parametrize("rows,cache", KINDS)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_see(rows, cache, what):
    """Keys and values that are not finite, within the chunk: rows before them are as if they were not there, rows that see them
    have what the formula gives."""
    c = Case([(150, 40), (70, 70)], 4, 2, 128, 16, rows, cache, seed=4)
    c.set(0, 130, v=what)
    c.set(1, 33, v=what)
    c.v[c.table[1, 3], 0, 5, 7] = what           # one element of one head
    c.upload().run().check()
    c = Case([(150, 40), (70, 70)], 4, 2, 128, 16, rows, cache, seed=5)
    c.set(0, 130, k=float("nan"), v=what)
    c.set(1, 33, k=float("nan"))
    c.upload().run()
    want = c.want()
    assert np.isfinite(want[0][:20]).all() and np.isnan(want[0][20:40]).all()
    c.check(want)
    c = Case([(150, 40)], 4, 2, 128, 16, rows, cache, seed=6)
    c.window = 30
    c.set(0, 100, v=what)                         # left behind by the window
    c.set(0, 119, k=what if np.isnan(what) else 1.0, v=what)
    c.upload().run().check()


@pytest.mark.parametrize("rows,cache", KINDS)
def test_magnitudes(rows, cache):
    """Scores of thousands, of either sign, all alike, and rows of zeros; large and tiny rows of q."""
    c = Case([(100, 4), (64, 4), (300, 4)], 4, 2, 64, 16, rows, cache, seed=7, spread=4.0)
    c.q[0] *= 40
    c.q[1] = 0
    c.q[2] *= 2.0 ** -12
    c.q[4] = -c.q[4] * 30
    if rows == "f32":
        c.q[5] *= 2.0 ** 40
        c.q[6] *= 2.0 ** -60
        c.q[7, 0, 0] = 2.0 ** 20
    c.upload().run().check()


def test_values_alike():
    """With one value everywhere the weights' roundings cancel."""
    c = Case([(777, 3)], 4, 2, 128, 16, "bf16", "bf16", seed=8)
    c.v[:] = 1.25
    c.upload().run()
    assert torch.all((c.out.float() - 1.25).abs() <= 1.25 * 2.0 ** -8)


@pytest.mark.parametrize("n", [63, 257, 1500])
def test_many_requests(n):
    rng = np.random.default_rng(n)
    requests = [(int(x), min(int(x), int(y))) for x, y in zip(rng.integers(0, 60, n), rng.integers(0, 3, n))]
    requests[n // 2] = (900, 1)
    c = Case(requests, 2, 1, 64, 16, "f32", "bf16", seed=n)
    c.upload().run().check()


def test_the_same_call_gives_the_same_bits():
    c = Case([(5000, 1), (900, 33), (70, 2)], 16, 2, 256, 16, "bf16", "bf16", seed=9).upload()
    first = c.run().out.clone()
    for _ in range(5):
        c.out.fill_(3.0)
        c.ws.fill_(0xFF)
        assert torch.equal(c.run().out, first)


def test_offsets_that_are_none():
    """Offsets past the rows, descending or negative reach nothing beside the outputs."""
    c = Case([(40, 4), (50, 4), (60, 4)], 4, 2, 64, 16, "bf16", "bf16", seed=10)
    for offsets, lengths in (([0, 100, 2, 2 ** 31 - 1], [40, 50, 60]), ([-5, 3, -2, 9], [40, -50, 2 ** 31 - 1]), ([12, 0, 12, 0], [1, 2, 3]),
                             ([2 ** 31 - 1, -2 ** 31, 5, 6], [10 ** 9, 50, 60])):
        c.upload(extra=2)
        c.do, c.dl = ints(offsets), ints(lengths)
        c.run()
        torch.cuda.synchronize()


def test_past_4_gib():
    """A cache whose pages 32 bits cannot count in bytes."""
    kv, dim, page = 8, 256, 256
    c = Case([(600, 2)], 16, kv, dim, page, "bf16", "bf16", seed=11)
    pages = 4300
    c.upload()
    k, v = (torch.full((pages, kv, page, dim), float("nan"), dtype=torch.bfloat16, device=gu.DEV) for _ in range(2))
    far = [pages - 1, 7, pages - 40]
    for at, p in zip(far, c.table[0]):
        k[at], v[at] = c.dk[p], c.dv[p]
    want = c.want()
    c.handle, c.dt = tb.KvCache(k, v), ints([far + [-1]])
    c.run().check(want)


def test_streams_and_graphs():
    """On another stream, on two at once with a workspace each, and captured: replayed while the request grows."""
    c = Case([(500, 1), (900, 1)], 16, 2, 256, 16, "bf16", "bf16", seed=12).upload()
    first = c.run().out.clone()
    torch.cuda.synchronize()
    d = Case([(2000, 1), (90, 20)], 16, 2, 256, 16, "bf16", "bf16", seed=13).upload()
    other = d.run().out.clone()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        c.out.zero_()
        d.out.zero_()
        torch.cuda.synchronize()
        c.run(stream=a)
        d.run(stream=b)
        torch.cuda.synchronize()
        assert torch.equal(c.out, first) and torch.equal(d.out, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for n in ((500, 900), (17, 880), (1, 1), (500, 899)):
        c.lengths = list(n)
        c.dl.copy_(ints(n))
        c.out.zero_()
        c.ws.fill_(0xFF)
        graph.replay()
        c.check()
        again = c.out.clone()
        torch.randn(1000, device=gu.DEV).sum().item()
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, again)


def test_refusals():
    c = Case([(40, 4)], 4, 2, 64, 16, "bf16", "bf16", seed=14).upload()
    good = dict(q=c.dq, cache=c.handle, table=c.dt, offsets=c.do, lengths=c.dl, scale=c.scale, out=c.out, ws=c.ws)
    for bad in (dict(q=c.dq.half()), dict(q=c.dq[:, :3]), dict(q=c.dq[0]), dict(q=c.dq.cpu()), dict(table=c.dt.long()), dict(offsets=c.do[:1]),
                dict(lengths=c.do), dict(out=c.out.float()), dict(out=c.out[:3]), dict(ws=c.ws[:100]), dict(ws=c.ws.float()), dict(scale=0.0),
                dict(scale=float("nan")), dict(window=-1), dict(gate=c.dq[:3]), dict(gate=c.dq[:, :2]), dict(gate=c.dq.int()), dict(out=c.dq)):
        with pytest.raises(tb.TbError) as e:
            tb.tb_attn_paged(**{**good, **bad})
        assert e.value.status == tb.TB_EINVAL, bad.keys()
    odd = torch.zeros(40, 2, 16, 96, dtype=torch.bfloat16, device=gu.DEV)
    q = torch.zeros(4, 4, 96, dtype=torch.bfloat16, device=gu.DEV)
    with pytest.raises(tb.TbError) as e:
        tb.tb_attn_paged(**{**good, "cache": tb.KvCache(odd, odd.clone()), "q": q, "out": q.clone()})
    assert e.value.status == tb.TB_EUNSUPPORTED
    assert torch.all(c.out == 77.0)


@pytest.mark.parametrize("rows,cache", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_chunks(dim, rows, cache):
    """Chunks of many tiles beside single tokens, a window, pages that are none, values that are not finite: the kernel for many rows
    at every width, its units cut by the borders of the workgroups' stretches."""
    say(f"chunks dim={dim} {rows}/{cache}")
    heads, kv = (6, 2) if dim < 256 else (5, 1)
    for window in (0, 77):
        c = Case([(331, 200), (9, 1), (64, 64), (700, 33), (1, 1)], heads, kv, dim, 32, rows, cache, seed=dim + window)
        c.window = window
        c.table[3, 4] = -1
        c.set(0, 250, v=float("nan"))
        c.set(0, 300, k=float("nan"))
        c.v[c.table[2, 1], 0, 3, 5] = float("inf")
        c.upload(extra=3).run().check()
        assert torch.all(c.out[c.tokens:] == 77.0)


@pytest.mark.parametrize("group", [1, 2, 5, 16, 17, 40])
def test_groups(group):
    """Heads of a kv head beside the tiles of 16 rows: fewer, as many, more, and more than one tile for a single token."""
    say(f"group {group}")
    Case([(300, 1), (45, 1), (0, 0)], group, 1, 64, 16, "bf16", "bf16", seed=group).upload().run().check()
    Case([(300, 9), (45, 45)], group * 2, 2, 64, 16, "f32", "f16", seed=group).upload().run().check()


def test_shared_pages_and_caches():
    """Requests that share pages, a cache whose keys are its values, and a query row that all rows share."""
    c = Case([(100, 1), (100, 1)], 4, 2, 64, 16, "bf16", "bf16", seed=21)
    c.table[1, :5] = c.table[0, :5]
    c.v = c.k.clone()
    c.q[1] = c.q[0]
    c.upload()
    c.handle = tb.KvCache(c.dk, c.dk)
    c.dq = c.dq[:1].expand(2, 4, 64)
    c.run().check()


def test_a_workspace_that_two_graphs_share():
    """Two captured calls of different shapes, one workspace, replayed in turn."""
    a = Case([(900, 1), (40, 1)], 16, 2, 256, 16, "bf16", "bf16", seed=22).upload()
    b = Case([(700, 90), (50, 3)], 6, 2, 128, 16, "f16", "f16", seed=23).upload()
    a.ws = b.ws = torch.full((max(a.ws.numel(), b.ws.numel()),), 0xFF, dtype=torch.uint8, device=gu.DEV)
    wants = a.want(), b.want()
    graphs = []
    for c in (a, b):
        c.run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.run()
    for turn in range(4):
        for c, g, w in zip((a, b), graphs, wants):
            c.out.zero_()
            g.replay()
            c.check(w)
            torch.randn(100, device=gu.DEV).sum().item()


def test_a_layer_as_it_is_used():
    """Prompt, then decoding, of two requests: plan -> fused projection -> rotation into the pages -> attention -> output
    projection, with the ternary products, against the same steps in 64 bits on the projections' own rows."""
    from ternary_weight_int8_tb_amd import synth
    heads, kv, dim, page, hidden = 4, 1, 64, 16, 256
    width = 2 * heads * dim + 2 * kv * dim
    wq = tb.Matrix.upload(synth.matrix(synth.FMT_TERNARY2, width, hidden, 5, 0, synth.T_GATE))
    wo = tb.Matrix.upload(synth.matrix(synth.FMT_TERNARY2, hidden, heads * dim, 5, 1, synth.T_DOWN))
    pages, columns = 12, 6
    cache = tb.KvCache(*(torch.full((pages, kv, page, dim), float("nan"), dtype=torch.bfloat16, device=gu.DEV) for _ in range(2)))
    rope = tb.Rope.make(32, base=10000.0)
    table = torch.full((2, columns), -1, dtype=torch.int32, device=gu.DEV)
    free, count = ints(np.arange(pages)[::-1].copy()), ints([pages])
    lengths, offsets = ints([0, 0]), ints([0, 0, 0])
    missing = ints([0])
    g = torch.Generator().manual_seed(1)
    scale = float(np.float32(dim ** -0.5))
    for fresh in ([19, 7], [1, 1], [1, 0], [1, 1], [0, 6]):
        t = sum(fresh)
        x = torch.randn(t, hidden, generator=g).to(gu.DEV)
        positions, slots = gu.i32_out(t), gu.i32_out(t)
        tb.tb_kv_plan(lengths, ints(fresh), page, pages, table, free, count, lengths, offsets, positions, slots, count, missing)
        fused = gu.f32_out(t, width)
        qx, dqx = gu.i8_out(t, hidden), gu.f32_out(t, hidden // 128)
        for r in range(0, t, 8):      # eight rows a call
            m = min(8, t - r)
            tb.tb_gemv_ternary_x(wq, x[r:r + m], qx[r:r + m], dqx[r:r + m].contiguous(), fused[r:r + m])
        fused *= 4.0
        view = (lambda at, n: fused[:, at:at + n * dim].view(t, n, dim))
        q, gate, k, v = view(0, heads), view(heads * dim, heads), view(2 * heads * dim, kv), view(2 * heads * dim + kv * dim, kv)
        q_out, out = gu.f32_out(t, heads, dim), gu.f32_out(t, heads, dim)
        tb.tb_rope_kv(q, k, v, rope, positions, slots, cache, q_out)
        ws = torch.empty(tb.tb_attn_paged_workspace_bytes(cache, heads, torch.float32, 2, t), dtype=torch.uint8, device=gu.DEV)
        tb.tb_attn_paged(q_out, cache, table, offsets, lengths, scale, out, ws, gate=gate)
        y = gu.f32_out(t, hidden)
        qh, dqh = gu.i8_out(t, heads * dim), gu.f32_out(t, heads * dim // 128)
        for r in range(0, t, 8):
            m = min(8, t - r)
            tb.tb_gemv_ternary_x(wo, out.view(t, -1)[r:r + m], qh[r:r + m], dqh[r:r + m].contiguous(), y[r:r + m])
        # the same steps in 64 bits
        ln, off, tab = (gu.host(z) for z in (lengths, offsets, table))
        assert int(gu.host(missing)[0]) == 0 and off[-1] == t and np.isfinite(gu.host(y)).all()
        pos, slot = gu.host(positions), gu.host(slots)
        for s in range(2):
            n = off[s + 1] - off[s]
            assert list(pos[off[s]:off[s + 1]]) == list(range(ln[s] - n, ln[s]))
        freq = rope.freq.cpu().numpy()
        for got, rows in ((q_out, q), (None, k)):
            want, size = plain_kv.rope(rows.double().cpu().numpy(), pos, freq, 1.0, False)
            if got is not None:
                assert np.all(np.abs(gu.host(got) - want) <= size * 9 * plain_kv.U)
            else:
                kept = cache.k.float().cpu().numpy()[slot // page, :, slot % page]
                assert np.all(np.abs(kept - want) <= size * 9 * plain_kv.U + 2.0 ** -8 * np.abs(want) * 1.001)
        assert np.array_equal(cache.v.float().cpu().numpy()[slot // page, :, slot % page], v.to(torch.bfloat16).float().cpu().numpy())
        want = plain_kv.attention(q_out.double().cpu().numpy(), cache.k.double().cpu().numpy(), cache.v.double().cpu().numpy(), tab, off, ln, scale,
                                  0, gate.double().cpu().numpy())
        assert np.all(np.abs(gu.host(out) - want[0]) <= plain_kv.attention_bound(*want, dim, "f32", "bf16"))
