"""An FFN of experts on MI355X: every pair's row has the bits of the single-matrix calls, and the
token's sum is that of the definition in 64 bits."""

from __future__ import annotations

import functools

import numpy as np
import pytest
import torch

import oracle
import ternary_weight_int8_tb_amd as tb
from tests import gpu_util as gu
from tests import plain
from tests.plain import U
from ternary_weight_int8_tb_amd import synth

pytestmark = pytest.mark.gpu

TERN, SIGN = synth.FMT_TERNARY2, synth.FMT_SIGN1


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield


class Layer:
    """E experts' packed matrices on the host, as Experts on the device, and one by one."""

    def __init__(self, fmt, experts, hidden, inter, seed):
        self.host = [synth.ffn_layer(seed, e, fmt, hidden=hidden, inter=inter) for e in range(experts)]
        for name in ("gate", "up", "down"):
            mats = [getattr(h, name) for h in self.host]
            setattr(self, name, tb.Experts.upload(mats))
            setattr(self, name + "_one", [tb.Matrix.upload(p) for p in mats])
        self.experts, self.hidden, self.inter, self.fmt = experts, hidden, inter, fmt


@functools.lru_cache(maxsize=None)
def layer_of(fmt, experts, hidden, inter):
    return Layer(fmt, experts, hidden, inter, 60)


class Run:
    """Poisoned buffers of one pass over `ids`."""

    def __init__(self, layer, q, dq, ids, weights=None, dtype=torch.float32):
        t, topk = ids.shape
        p = t * topk
        self.layer, self.q, self.dq, self.topk = layer, gu.dev(q), gu.dev(dq), topk
        self.ids = gu.dev(ids.astype(np.int32))
        self.weights = gu.dev(weights if weights is not None else np.ones((t, topk), np.float32))
        self.offsets, self.order = gu.i32_out(layer.experts + 1), gu.i32_out(p)
        self.h, self.qh, self.dqh = gu.f32_out(p, layer.inter), gu.i8_out(p, layer.inter), gu.f32_out(p, layer.inter // 128)
        self.y = gu.f32_out(p, layer.hidden)
        self.out = torch.full((t, layer.hidden), float("nan"), dtype=dtype, device=gu.DEV)

    def launch(self, stream=None):
        w = self.layer
        tb.tb_moe_plan(self.ids, w.experts, self.offsets, self.order, stream)
        tb.tb_moe_gateup_silu(w.gate, w.up, self.q, self.dq, self.topk, self.offsets, self.order, self.h, self.qh, self.dqh, stream)
        tb.tb_moe_down(w.down, self.qh, self.dqh, self.offsets, self.order, self.y, stream)
        tb.tb_moe_combine(self.y, self.weights, self.ids, w.experts, self.out, stream)
        return self


def rows(t, hidden, seed):
    x = synth.normal_rows(t, hidden, seed, 0)
    return oracle.default().rotate_quant(x)


def plan_of(ids, experts):
    flat = ids.reshape(-1)
    order = [p for e in range(experts) for p in np.nonzero(flat == e)[0]]
    counts = [(flat == e).sum() for e in range(experts)]
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), np.array(order, np.int32)


def check(run, ids):
    """Plan, rows and sums against the single-matrix calls (in parts of up to 32 rows)."""
    w = run.layer
    offsets, order = plan_of(ids, w.experts)
    assert np.array_equal(gu.host(run.offsets), offsets)
    got = gu.host(run.order)
    assert np.array_equal(got[:len(order)], order) and (got[len(order):] == gu.POISON_I32).all()
    qh, dqh, y = gu.host(run.qh), gu.host(run.dqh), gu.host(run.y)
    for e in range(w.experts):
        for a in range(offsets[e], offsets[e + 1], 32):
            b = min(a + 32, offsets[e + 1])
            pairs = order[a:b]
            token = torch.from_numpy((pairs // run.topk).astype(np.int64)).to(gu.DEV)
            m = b - a
            h, q2, dq2, y2 = gu.f32_out(m, w.inter), gu.i8_out(m, w.inter), gu.f32_out(m, w.inter // 128), gu.f32_out(m, w.hidden)
            tb.tb_ffn_gateup_silu_batch(w.gate_one[e], w.up_one[e], run.q[token].contiguous(), run.dq[token].contiguous(), h)
            tb.tb_ffn_down_batch(w.down_one[e], h, q2, dq2, y2)
            assert np.array_equal(qh[a:b], gu.host(q2)), f"qh, expert {e}"
            assert dqh[a:b].tobytes() == gu.host(dq2).tobytes(), f"dqh, expert {e}"
            assert y[pairs].tobytes() == gu.host(y2).tobytes(), f"y, expert {e}"
    used = int(offsets[-1])
    assert (qh[used:] == gu.POISON_I8).all() and np.isnan(dqh[used:]).all()
    flat = ids.reshape(-1)
    dropped = (flat < 0) | (flat >= w.experts)
    assert np.isnan(y[dropped]).all() and not np.isnan(y[~dropped]).any()
    # the sum, in 64 bits: topk products and sums in fp32, then one rounding to the output's type
    terms = np.where(dropped[:, None], 0.0, gu.host(run.weights).reshape(-1, 1).astype(np.float64) * y)
    terms = terms.reshape(ids.shape[0], run.topk, -1)
    want, size = terms.sum(1), np.abs(terms).sum(1)
    tol = (run.topk + 1) * U * size + torch.finfo(run.out.dtype).eps / 2 * (1 + 1e-3) * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(run.out.double().cpu().numpy() - want) <= tol)


def ids_of(kind, t, topk, experts, seed):
    rng = np.random.default_rng(seed)
    if kind == "distinct":
        return np.stack([rng.permutation(experts)[:topk] for _ in range(t)])
    if kind == "one":                       # all pairs to one expert
        return np.full((t, topk), experts - 1)
    if kind == "dropped":
        ids = rng.integers(0, experts, (t, topk))
        ids[rng.random((t, topk)) < 0.4] = -1
        ids.reshape(-1)[::7] = experts      # just past the last
        ids[0] = -(2 ** 31)
        return ids
    if kind == "none":
        return np.full((t, topk), -1)
    return rng.integers(0, experts, (t, topk))   # repeats allowed


@pytest.mark.parametrize("fmt", [TERN, SIGN])
@pytest.mark.parametrize("t,topk,experts,hidden,inter", [
    (1, 1, 1, 128, 128), (1, 4, 8, 256, 128), (3, 2, 5, 384, 256), (17, 2, 3, 640, 384), (40, 4, 70, 256, 128),
    (65, 1, 2, 1152, 640), (130, 8, 8, 2048, 1024), (300, 3, 4, 1408, 2176)])
@pytest.mark.parametrize("kind", ["distinct", "one", "dropped", "none", "any"])
def test_moe(fmt, t, topk, experts, hidden, inter, kind):
    print(f"moe fmt={fmt} t={t} topk={topk} E={experts} {hidden}x{inter} {kind}", flush=True)
    layer = layer_of(fmt, experts, hidden, inter)
    q, dq = rows(t, hidden, 61)
    ids = ids_of(kind, t, topk, experts, 62)
    weights = np.random.default_rng(63).standard_normal((t, topk)).astype(np.float32)
    check(Run(layer, q, dq, ids, weights).launch(), ids)


@pytest.mark.parametrize("fmt", [TERN, SIGN])
def test_moe_long_rows(fmt):
    """k over several parts of the workgroup's LDS, with a last step that is not full."""
    layer = Layer(fmt, 2, 128 * 75, 128 * 69, 64)
    q, dq = rows(9, layer.hidden, 65)
    ids = ids_of("distinct", 9, 2, 2, 66)
    check(Run(layer, q, dq, ids).launch(), ids)


@pytest.mark.parametrize("fmt", [TERN, SIGN])
@pytest.mark.parametrize("kind", ["distinct", "one", "dropped"])
def test_moe_long_rows_of_many_pairs(fmt, kind):
    layer = layer_of(fmt, 2, 128 * 37, 128 * 21)
    t = 130
    q, dq = rows(t, layer.hidden, 98)
    ids = ids_of(kind, t, 2, 2, 99)
    check(Run(layer, q, dq, ids).launch(), ids)


@pytest.mark.parametrize("fmt", [TERN, SIGN])
def test_moe_against_the_oracle(fmt):
    layer = Layer(fmt, 3, 512, 256, 67)
    q, dq = rows(11, 512, 68)
    ids = ids_of("distinct", 11, 2, 3, 69)
    run = Run(layer, q, dq, ids).launch()
    qh, dqh, y = gu.host(run.qh), gu.host(run.dqh), gu.host(run.y)
    offsets, order = plan_of(ids, 3)
    for e in range(3):
        w = plain.weights(layer.host[e].down)
        for s in range(offsets[e], offsets[e + 1]):
            v = qh[s].astype(np.float64).reshape(-1, 128) * dqh[s].astype(np.float64)[:, None]
            terms = np.einsum("bi,nbi->nb", v, w)
            assert np.all(np.abs(y[order[s]] - terms.sum(1)) <= 1e-4 * np.abs(terms).sum(1))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [1, 7, 128, 516])
def test_combine(n, dtype):
    t, topk, experts = 19, 3, 4
    rng = np.random.default_rng(70)
    ids = ids_of("dropped", t, topk, experts, 71)
    y = rng.standard_normal((t * topk, n)).astype(np.float32)
    flat = ids.reshape(-1)
    dropped = (flat < 0) | (flat >= experts)
    y[dropped] = np.nan
    weights = rng.standard_normal((t, topk)).astype(np.float32)
    weights.reshape(-1)[dropped] = np.inf
    out = torch.full((t, n), float("nan"), dtype=dtype, device=gu.DEV)
    tb.tb_moe_combine(gu.dev(y), gu.dev(weights), gu.dev(ids.astype(np.int32)), experts, out)
    terms = np.where(dropped[:, None], 0.0, np.where(dropped, 0, weights.reshape(-1))[:, None].astype(np.float64) * np.nan_to_num(y))
    terms = terms.reshape(t, topk, n)
    want, size = terms.sum(1), np.abs(terms).sum(1)
    tol = (topk + 1) * U * size + torch.finfo(dtype).eps / 2 * (1 + 1e-3) * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("pairs_topk_experts", [(1, 1, 1), (63, 1, 2), (64, 1, 300), (65, 1, 1000), (5000, 7, 64), (3, 5, 65536)])
def test_plan(pairs_topk_experts):
    t, topk, experts = pairs_topk_experts
    rng = np.random.default_rng(t)
    ids = rng.integers(-2, experts + 2, (t, topk)).astype(np.int32)
    offsets, order = gu.i32_out(experts + 1), gu.i32_out(t * topk)
    tb.tb_moe_plan(gu.dev(ids), experts, offsets, order)
    flat = ids.reshape(-1)
    kept = np.nonzero((flat >= 0) & (flat < experts))[0]
    want = kept[np.argsort(flat[kept], kind="stable")]
    got = gu.host(order)
    assert np.array_equal(got[:len(want)], want) and (got[len(want):] == gu.POISON_I32).all()
    counts = np.bincount(flat[kept], minlength=experts)
    assert np.array_equal(gu.host(offsets), np.concatenate([[0], np.cumsum(counts)]))


@pytest.mark.parametrize("t", [50, 150])   # tiles of few and of many pairs
def test_moe_graph_and_streams(t):
    """A captured pass follows its inputs from replay to replay; two layers run on two streams at once."""
    layer = Layer(TERN, 6, 512, 256, 72)
    topk = 2
    q, dq = rows(t, 512, 73)
    run = Run(layer, q, dq, ids_of("any", t, topk, 6, 74))
    run.launch()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run.launch()
    for r in range(3):
        ids = ids_of("dropped" if r == 1 else "any", t, topk, 6, 80 + r)
        run.ids.copy_(gu.dev(ids.astype(np.int32)))
        for b in (run.y, run.dqh, run.out):
            b.fill_(float("nan"))
        run.qh.fill_(gu.POISON_I8)
        run.order.fill_(gu.POISON_I32)
        graph.replay()
        check(run, ids)
    ids = [ids_of("any", t, topk, 6, 90 + r) for r in range(2)]
    runs = [Run(layer, q, dq, i) for i in ids]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for run, s in zip(runs, streams):
            run.launch(s)
    torch.cuda.synchronize()
    for run, i in zip(runs, ids):
        check(run, i)


def test_norm_route_experts():
    """The operators as a decoder block uses them: norm, experts, sum, and the next norm adds it."""
    layer = Layer(TERN, 4, 512, 256, 75)
    t, topk, hidden = 21, 2, 512
    g = torch.Generator().manual_seed(76)
    x, res = (torch.randn(t, hidden, generator=g).bfloat16().to(gu.DEV) for _ in range(2))
    gamma = (1 + 0.2 * torch.randn(hidden, generator=g)).to(gu.DEV)
    s, normed = torch.empty_like(x), torch.empty_like(x)
    q, dq = gu.i8_out(t, hidden), gu.f32_out(t, hidden // 128)
    tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-6, s, normed, q, dq)
    router = torch.randn(hidden, 4, generator=g).to(gu.DEV)
    top, ids = torch.topk(normed.float() @ router, topk, dim=1)
    run = Run(layer, gu.host(q), gu.host(dq), ids.cpu().numpy(), torch.softmax(top, 1).cpu().numpy(), torch.bfloat16)
    run.launch()
    check(run, ids.cpu().numpy())
    q2, dq2, s2 = gu.i8_out(t, hidden), gu.f32_out(t, hidden // 128), torch.empty_like(x)
    tb.tb_add_rmsnorm_quant_i8(run.out, s, gamma, 1e-6, s2, None, q2, dq2)
    assert torch.equal(s2, (run.out.float() + s.float()).bfloat16())
    # against the dense definition: the chain's int8 and bf16 roundings leave a few per cent
    v = (q.double().view(t, -1, 128) * dq.double()[..., None]).view(t, -1).cpu().numpy()
    want = np.zeros((t, hidden))
    for e, w in enumerate(layer.host):
        gate, up, down = (plain.weights(m).reshape(m.n, -1) for m in (w.gate, w.up, w.down))
        gg = v @ gate.T
        h = gg / (1 + np.exp(-gg)) * (v @ up.T)
        h = (h.reshape(t, -1, 128) @ (plain.hadamard() / np.sqrt(128))).reshape(t, -1)
        pick = (ids.cpu().numpy() == e) * torch.softmax(top, 1).cpu().numpy()
        want += pick.sum(1, keepdims=True) * (h @ down.T)
    got = run.out.double().cpu().numpy()
    assert np.linalg.norm(got - want) < 0.03 * np.linalg.norm(want)


@pytest.mark.parametrize("fmt", [TERN, SIGN])
@pytest.mark.parametrize("t", [7, 90])   # tiles of few and of many pairs
def test_every_int8_value(fmt, t):
    """Rows that no quantiser made: all 256 values of a byte."""
    layer = layer_of(fmt, 3, 640, 384)
    rng = np.random.default_rng(83)
    q = rng.integers(-128, 128, (t, 640)).astype(np.int8)
    q[0, :256] = np.arange(-128, 128)
    q[-1] = -128
    dq = rng.standard_normal((t, 5)).astype(np.float32)
    dq[t // 2] = 0.0
    ids = ids_of("any", t, 2, 3, 84)
    check(Run(layer, q, dq, ids).launch(), ids)


@pytest.mark.parametrize("fmt", [TERN, SIGN])
@pytest.mark.parametrize("t", [7, 90])
@pytest.mark.parametrize("k", [640, 1152])   # 5 and 9 blocks: the last step is not full
def test_scales_that_are_not_finite_stay_in_their_row(fmt, t, k):
    host = [synth.ffn_layer(85, e, fmt, hidden=256, inter=k).down for e in range(3)]
    ids = ids_of("any", t, 2, 3, 86)
    offsets, order = plan_of(ids, 3)
    qh, dqh = rows(2 * t, k, 87)
    out = []
    for plant in (False, True):
        w = tb.Experts.upload(host)
        if plant:
            bits = w.scales.view(torch.float16)
            bits[:, 0, 0] = float("inf")    # behind the last row of the expert before
            bits[:, 7, 0] = float("-inf")
            bits[:, 100, 0] = float("nan")
            bits[:, 255, -1] = float("inf")
        y = gu.f32_out(2 * t, 256)
        tb.tb_moe_down(w, gu.dev(qh), gu.dev(dqh), gu.dev(offsets), gu.dev(order), y)
        out.append(gu.host(y))
    hit = [0, 7, 100, 255]
    assert not np.isfinite(out[1][:, hit]).any()
    assert np.delete(out[1], hit, 1).tobytes() == np.delete(out[0], hit, 1).tobytes()


@pytest.mark.parametrize("fmt", [TERN, SIGN])
@pytest.mark.parametrize("t", [7, 90])
def test_rows_that_are_not_finite_stay_alone(fmt, t):
    """A token whose scales are NaN or infinite changes no other token's rows."""
    layer = layer_of(fmt, 3, 640, 384)
    q, dq = rows(t, 640, 95)
    ids = ids_of("any", t, 2, 3, 96)
    clean = Run(layer, q, dq, ids).launch()
    bad = dq.copy()
    bad[2], bad[t - 1, 0] = np.nan, np.inf
    run = Run(layer, q, bad, ids).launch()
    good = [x for x in range(t) if x not in (2, t - 1)]
    assert torch.equal(run.out[good], clean.out[good])


def test_two_layers_at_once():
    """Two streams, each with its own buffers, on the same experts."""
    layer = layer_of(TERN, 8, 2048, 1024)
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for x, t in enumerate((3, 60)):
        q, dq = rows(t, 2048, 88 + x)
        ids = ids_of("dropped", t, 4, 8, 90 + x)
        runs.append((Run(layer, q, dq, ids), ids))
    torch.cuda.synchronize()
    for _ in range(3):
        for (run, _), s in zip(runs, streams):
            run.launch(s)
    torch.cuda.synchronize()
    for run, ids in runs:
        check(run, ids)


def test_offsets_that_are_no_plan():
    """Lists that overlap, so that there are more slots than pairs."""
    layer = layer_of(TERN, 3, 640, 384)
    for t in (9, 90):
        q, dq = rows(t, 640, 92)
        run = Run(layer, q, dq, ids_of("any", t, 2, 3, 93))
        for bad in ([0, 2 * t, 0, 2 * t], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1], [5, 5, 5, 5]):
            run.offsets.copy_(torch.tensor(bad, dtype=torch.int32))
            run.order.copy_(torch.arange(2 * t, dtype=torch.int32).flip(0))
            tb.tb_moe_gateup_silu(layer.gate, layer.up, run.q, run.dq, 2, run.offsets, run.order, run.h, run.qh, run.dqh)
            tb.tb_moe_down(layer.down, run.qh, run.dqh, run.offsets, run.order, run.y)
    torch.cuda.synchronize()


def test_large_offsets():
    """Codes, activations and rows of outputs past 4 GiB."""
    experts, n, k, pairs = 66, 8320, 32768, 132000
    gen = torch.Generator(device=gu.DEV).manual_seed(94)
    codes = torch.randint(0, 256, (experts, n, k // 128, 32), dtype=torch.uint8, device=gu.DEV, generator=gen)
    scales = torch.rand((experts, n, k // 128), device=gu.DEV, generator=gen).half()
    qh = torch.randint(-127, 128, (pairs, k), dtype=torch.int8, device=gu.DEV, generator=gen)
    dqh = torch.rand((pairs, k // 128), device=gu.DEV, generator=gen)
    ids = torch.randint(0, experts, (pairs, 1), dtype=torch.int32, device=gu.DEV, generator=gen)
    offsets, order = gu.i32_out(experts + 1), gu.i32_out(pairs)
    y = torch.empty((pairs, n), device=gu.DEV)
    tb.tb_moe_plan(ids, experts, offsets, order)
    tb.tb_moe_down(tb.Experts(codes, scales, TERN), qh, dqh, offsets, order, y)
    lists = offsets.tolist()
    for e in (0, experts // 2, experts - 1):
        one = tb.Matrix(codes[e], scales[e].view(torch.int16), n, k, TERN)
        a, b = lists[e], lists[e + 1]
        slots = torch.tensor([a, a + 1, (a + b) // 2, b - 1], device=gu.DEV)
        want = gu.f32_out(4, n)
        tb.tb_gemv_ternary(one, qh[slots].contiguous(), dqh[slots].contiguous(), want)
        assert torch.equal(y[order[slots].long()], want), f"expert {e}"


def test_more_items_than_a_launch_holds():
    """Over 2^20 workgroups: 40000 experts of 32 row groups, about one pair each."""
    experts, n, k, pairs = 40000, 4096, 128, 40000
    gen = torch.Generator(device=gu.DEV).manual_seed(97)
    codes = torch.randint(0, 256, (experts, n, 1, 16), dtype=torch.uint8, device=gu.DEV, generator=gen)
    scales = torch.rand((experts, n, 1), device=gu.DEV, generator=gen).half()
    qh = torch.randint(-127, 128, (pairs, k), dtype=torch.int8, device=gu.DEV, generator=gen)
    dqh = torch.rand((pairs, 1), device=gu.DEV, generator=gen)
    ids = torch.randint(0, experts, (pairs, 1), dtype=torch.int32, device=gu.DEV, generator=gen)
    offsets, order = gu.i32_out(experts + 1), gu.i32_out(pairs)
    y = gu.f32_out(pairs, n)
    tb.tb_moe_plan(ids, experts, offsets, order)
    tb.tb_moe_down(tb.Experts(codes, scales, SIGN), qh, dqh, offsets, order, y)
    lists = gu.host(offsets)
    assert np.array_equal(lists, np.searchsorted(np.sort(gu.host(ids)[:, 0]), np.arange(experts + 1)))
    assert not torch.isnan(y).any()
    for e in np.nonzero(np.diff(lists))[0][[0, 1000, 20000, -1]]:
        one = tb.Matrix(codes[e], scales[e].view(torch.int16), n, k, SIGN)
        slot = int(lists[e])
        want = gu.f32_out(1, n)
        tb.tb_gemv_ternary(one, qh[slot:slot + 1].clone(), dqh[slot:slot + 1].clone(), want)
        assert torch.equal(y[order[slot].long()], want[0]), f"expert {e}"


def test_offsets_out_of_range_are_cut():
    """A plan that did not come from tb_moe_plan touches nothing past the arrays."""
    layer = Layer(TERN, 3, 256, 128, 77)
    q, dq = rows(6, 256, 78)
    run = Run(layer, q, dq, ids_of("any", 6, 2, 3, 79))
    run.offsets.copy_(torch.tensor([-5, 7, 4, 1000], dtype=torch.int32))
    run.order.copy_(torch.tensor([0, 11, 12, -1, 2 ** 31 - 1, -2 ** 31, 3, 4, 5, 6, 7, 8], dtype=torch.int32))
    tb.tb_moe_gateup_silu(layer.gate, layer.up, run.q, run.dq, 2, run.offsets, run.order, run.h, run.qh, run.dqh)
    tb.tb_moe_down(layer.down, run.qh, run.dqh, run.offsets, run.order, run.y)
    torch.cuda.synchronize()
    assert not torch.isnan(run.y[[0, 11, 3, 4, 5, 6, 7, 8]]).any()


def test_binding_refusals():
    layer = Layer(TERN, 2, 256, 128, 80)
    q, dq = rows(3, 256, 81)
    r = Run(layer, q, dq, ids_of("any", 3, 2, 2, 82))

    def refuse(fn, *a):
        with pytest.raises(tb.TbError):
            fn(*a)
    refuse(tb.tb_moe_plan, r.ids.long(), 2, r.offsets, r.order)
    refuse(tb.tb_moe_plan, r.ids, 3, r.offsets, r.order)
    refuse(tb.tb_moe_plan, r.ids, 2, r.offsets, r.order[:5])
    refuse(tb.tb_moe_plan, r.ids.t(), 2, r.offsets, r.order)
    w = layer
    refuse(tb.tb_moe_gateup_silu, w.gate, w.down, r.q, r.dq, 2, r.offsets, r.order, r.h, r.qh, r.dqh)
    refuse(tb.tb_moe_gateup_silu, w.gate, w.up, r.q, r.dq, 3, r.offsets, r.order, r.h, r.qh, r.dqh)
    refuse(tb.tb_moe_gateup_silu, w.gate, w.up, r.q[:, :128].contiguous(), r.dq, 2, r.offsets, r.order, r.h, r.qh, r.dqh)
    refuse(tb.tb_moe_gateup_silu, w.gate, w.up, r.q, r.dq, 2, r.offsets, r.order, r.h, r.qh.to(torch.uint8), r.dqh)
    refuse(tb.tb_moe_down, w.down, r.qh, r.dqh, r.offsets, r.order, r.y[:5])
    refuse(tb.tb_moe_down, w.gate, r.qh, r.dqh, r.offsets, r.order, r.y)
    refuse(tb.tb_moe_combine, r.y, r.weights.double(), r.ids, 2, r.out)
    refuse(tb.tb_moe_combine, r.y, r.weights, r.ids, 2, r.out[:, :255])
    refuse(tb.Experts, w.gate.codes, w.gate.scales, synth.FMT_SIGN1)
    refuse(tb.Experts, w.gate.codes[:1], w.gate.scales, TERN)
    refuse(tb.Experts, w.gate.codes, w.gate.scales.float(), TERN)
    assert np.isnan(gu.host(r.y)).all() and np.isnan(gu.host(r.h)).all()


@pytest.mark.parametrize("fmt", [TERN, SIGN])
@pytest.mark.parametrize("t", [7, 90])   # tiles of few and of many pairs
def test_rows_that_are_not_finite_say_so(fmt, t):
    """What is not finite in a token's scales is not finite in its sum either."""
    layer = layer_of(fmt, 3, 640, 384)
    q, dq = rows(t, 640, 100)
    ids = ids_of("any", t, 2, 3, 101)
    dq[1], dq[2, 4], dq[t - 1, 0] = np.nan, np.nan, np.inf
    run = Run(layer, q, dq, ids).launch()
    bad = [1, 2, t - 1]
    assert not torch.isfinite(run.out[bad]).any()
    offsets, order = plan_of(ids, 3)
    slots = np.isin(order // 2, bad)
    assert np.isnan(gu.host(run.dqh)[slots]).all() and not gu.host(run.qh)[slots].any()
    assert np.isfinite(gu.host(run.dqh)[~slots]).all() and np.isfinite(np.delete(gu.host(run.out), bad, 0)).all()


@pytest.mark.parametrize("fmt", [TERN, SIGN])
@pytest.mark.parametrize("t", [7, 90])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_block_of_h_that_is_not_finite(fmt, t, value):
    """One value of h that is not finite marks its block of 128, and no other block's bits change."""
    host = [synth.ffn_layer(102, e, fmt, hidden=640, inter=384) for e in range(3)]
    gate, up = (tb.Experts.upload([getattr(w, n) for w in host]) for n in ("gate", "up"))
    q, dq = rows(t, 640, 103)
    ids = ids_of("any", t, 2, 3, 104)
    offsets, order = plan_of(ids, 3)
    out = []
    for plant in (False, True):
        if plant:
            up.scales.view(torch.float16)[1, 128 + 77, 2] = value   # expert 1, column 205: block 1 of h
        h, qh, dqh = gu.f32_out(2 * t, 384), gu.i8_out(2 * t, 384), gu.f32_out(2 * t, 3)
        tb.tb_moe_gateup_silu(gate, up, gu.dev(q), gu.dev(dq), 2, gu.dev(offsets), gu.dev(order), h, qh, dqh)
        out.append((gu.host(qh).reshape(2 * t, 3, 128), gu.host(dqh)))
    hit = np.zeros((2 * t, 3), bool)
    hit[offsets[1]:offsets[2], 1] = True
    assert hit.any() and np.isnan(out[1][1][hit]).all() and not out[1][0][hit].any()
    assert out[1][0][~hit].tobytes() == out[0][0][~hit].tobytes() and out[1][1][~hit].tobytes() == out[0][1][~hit].tobytes()


@pytest.mark.parametrize("t", [9, 90])
def test_offsets_that_are_no_plan_write_inside_the_outputs(t):
    """The outputs lie between poisoned rows of larger arrays, which stay as they are."""
    layer = layer_of(TERN, 3, 640, 384)
    q, dq = rows(t, 640, 105)
    p, pad = 2 * t, 16
    for bad in ([0, 2 * t, 0, 2 * t], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1], [5, 5, 5, 5], [-5, 7, 4, 1000]):
        offsets = gu.dev(np.array(bad, np.int32))
        order = gu.dev(np.random.default_rng(106).integers(-p, 2 * p, p).astype(np.int32))
        whole = {"h": gu.f32_out(p + 2 * pad, 384), "qh": gu.i8_out(p + 2 * pad, 384), "dqh": gu.f32_out((p + 2 * pad) * 4, 3),
                 "y": gu.f32_out(p + 2 * pad, 640)}
        part = {n: a[pad:pad + p] for n, a in whole.items()}
        part["dqh"] = whole["dqh"][4 * pad:4 * pad + p]
        tb.tb_moe_gateup_silu(layer.gate, layer.up, gu.dev(q), gu.dev(dq), 2, offsets, order, part["h"], part["qh"], part["dqh"])
        tb.tb_moe_down(layer.down, part["qh"], part["dqh"], offsets, order, part["y"])
        for n, a in whole.items():
            lo = 4 * pad if n == "dqh" else pad
            for around in (a[:lo], a[lo + p:]):
                assert (gu.host(around) == gu.POISON_I8).all() if n == "qh" else np.isnan(gu.host(around)).all(), (n, bad)
