"""Refusals of the calls around the paged cache, and the binding's frequencies, without a GPU: no call here reaches a launch."""

import ctypes
import math
import os

import numpy as np
import pytest

import ternary_weight_int8_tb_amd as tb
from tests import plain_kv
from ternary_weight_int8_tb_amd import build as tb_build

A = [(i + 1) << 32 for i in range(16)]      # fake 16-byte aligned addresses, 4 GiB apart
LAST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(tb.LIB_PATH):
        tb_build.build()
    return tb.lib()


def common(call, arrays, sizes=(), apart=()):
    """Null, misaligned and overlapping arrays. arrays: name -> (address, is an output); `apart`: pairs that may be one array."""
    for n, (a, out) in arrays.items():
        assert call(**{n: None}) == tb.TB_EINVAL, n
        assert call(**{n: a + 4}) == tb.TB_EALIGN, n
        for n2, (a2, out2) in arrays.items():
            if n != n2 and (out or out2) and (n, n2) not in apart:
                assert call(**{n: a2}) == tb.TB_EINVAL, (n, n2)
    for n, values in sizes:
        for v in values:
            assert call(**{n: v}) == tb.TB_EINVAL, (n, v)


PLAN = ("context", "fresh", "table", "free_list", "count", "lengths", "offsets", "positions", "slots", "left", "missing")


def plan_call(L):
    def call(requests=4, rows=64, page=16, pages=512, width=32, **a):
        a = {**dict(zip(PLAN, A)), **a}
        return L.tb_kv_plan(a["context"], a["fresh"], requests, rows, page, pages, a["table"], width, a["free_list"], a["count"],
                            a["lengths"], a["offsets"], a["positions"], a["slots"], a["left"], a["missing"], None)
    return call


def test_plan(L):
    call = plan_call(L)
    outs = set(PLAN) - {"context", "fresh", "count"}
    may = {("lengths", "context"), ("left", "count"), ("context", "lengths"), ("count", "left")}
    common(call, {n: (a, n in outs) for n, a in zip(PLAN, A)},
           [("requests", (0, -1)), ("rows", (0, -1)), ("width", (0, -1)), ("pages", (0, -1)), ("page", (0, 8, 17, 48, 512, -16))], may)
    assert call(requests=8, lengths=A[0] + 16) == tb.TB_EINVAL   # neither context itself nor apart from it
    assert call(left=A[5], lengths=A[5]) == tb.TB_EINVAL
    assert call(lengths=A[0], left=A[0]) == tb.TB_EINVAL
    assert call(pages=1 << 27) == tb.TB_EINVAL             # pages * page past 31 bits


def test_plan_limits(L):
    call = plan_call(L)
    far = dict(zip(PLAN, [(i + 1) << 48 for i in range(11)]))
    assert call(requests=16385, **far) == tb.TB_EUNSUPPORTED
    assert call(rows=1 << 30, **far) == tb.TB_EUNSUPPORTED
    assert call(rows=LAST, requests=LAST, width=LAST, **far) == tb.TB_EUNSUPPORTED
    assert call(requests=16384, width=1 << 16, **far) == tb.TB_EUNSUPPORTED
    assert call(width=(1 << 26) + 1, **far) == tb.TB_EUNSUPPORTED


def heads(base, row=9216, head=256, n=16, dtype=tb.TB_BF16):
    return tb.CHeads(base, row, head, n, dtype)


def cache(k=A[8], v=A[9], pages=64, kv=2, page=16, dim=256, dtype=tb.TB_BF16):
    return tb.CKvCache(k, v, pages, kv, page, dim, dtype)


def ref(x):
    return None if x is None else ctypes.byref(x)


def rope_call(L):
    def call(q=0, k=0, v=0, tokens=3, dim=256, rope=0, positions=A[3], slots=A[4], c=0, q_out=A[5], dtype=tb.TB_BF16):
        q = heads(A[0]) if q == 0 else q
        k = heads(A[1], n=2) if k == 0 else k
        v = heads(A[2], n=2) if v == 0 else v
        rope = tb.CRope(A[6], 64, 0, 1.0) if rope == 0 else rope
        c = cache() if c == 0 else c
        return L.tb_rope_kv(ref(q), ref(k), ref(v), tokens, dim, ref(rope), positions, slots, ref(c), q_out, dtype, None)
    return call


def test_rope(L):
    call = rope_call(L)
    common(call, {"positions": (A[3], False), "slots": (A[4], False), "q_out": (A[5], True)},
           [("tokens", (0, -1)), ("dim", (0, 8, 100, 528, 128)), ("dtype", (-1, 3))])
    for n, x in (("q", A[0]), ("k", A[1]), ("v", A[2])):
        mk = (lambda **a: heads(**{"base": x, "n": 16 if n == "q" else 2, **a}))
        assert call(**{n: mk(base=None)}) == tb.TB_EINVAL
        assert call(**{n: mk(base=x + 8)}) == tb.TB_EALIGN
        for bad in (dict(row=9217), dict(row=-8), dict(head=12), dict(head=-256), dict(n=0), dict(n=65537), dict(dtype=3), dict(dtype=tb.TB_F32),
                    dict(row=1 << 60), dict(head=1 << 62)):
            assert call(**{n: mk(**bad)}) == tb.TB_EINVAL, (n, bad)
        assert call(**{n: None}) == tb.TB_EINVAL              # q_out without q; k without v
        assert call(q_out=x) == tb.TB_EINVAL
    for bad in (dict(pages=0), dict(kv=0), dict(kv=65537), dict(page=8), dict(page=24), dict(dim=128), dict(dtype=tb.TB_F32), dict(k=None), dict(v=A[8]),
                dict(k=A[0]), dict(v=A[5]), dict(k=A[3]), dict(pages=1 << 27), dict(kv=3)):
        assert call(c=cache(**bad)) == tb.TB_EINVAL, bad
    assert call(c=cache(v=A[9] + 8)) == tb.TB_EALIGN
    for rot, layout in ((0, 0), (8, 0), (24, 1), (272, 0), (-16, 0), (64, 2), (64, -1)):
        assert call(rope=tb.CRope(A[6], rot, layout, 1.0)) == tb.TB_EINVAL
    assert call(rope=tb.CRope(None, 64, 0, 1.0)) == tb.TB_EINVAL
    assert call(rope=tb.CRope(A[6] + 8, 64, 0, 1.0)) == tb.TB_EALIGN
    assert call(q=None, q_out=None, k=None, v=None, slots=None, c=None) == tb.TB_EINVAL     # nothing to do
    assert call(q=None) == tb.TB_EINVAL and call(c=None) == tb.TB_EINVAL and call(k=None) == tb.TB_EINVAL
    far = dict(q=heads(1 << 50), k=heads(2 << 50, n=2), v=heads(3 << 50, n=2), positions=4 << 50, slots=5 << 50, q_out=6 << 50)
    assert call(tokens=1 << 24, **far) == tb.TB_EUNSUPPORTED


ATTN = ("table", "offsets", "lengths", "out", "ws")


def attn_call(L):
    def call(q=0, gate=None, c=0, width=64, requests=3, tokens=40, scale=0.0625, window=0, ws_bytes=1 << 30, **a):
        a = {**dict(zip(ATTN, A[1:6])), **a}
        q = heads(A[0]) if q == 0 else q
        c = cache() if c == 0 else c
        return L.tb_attn_paged(ref(q), ref(gate), ref(c), a["table"], width, a["offsets"], a["lengths"], requests, tokens, scale, window,
                               a["out"], a["ws"], ws_bytes, None)
    return call


def test_attention(L):
    call = attn_call(L)
    common(call, {n: (a, n in ("out", "ws")) for n, a in zip(ATTN, A[1:6])},
           [("requests", (0, -1)), ("tokens", (0, -1)), ("width", (0, -1)), ("window", (-1,)),
            ("scale", (0.0, -1.0, float("nan"), float("inf"))), ("ws_bytes", (0, 4096))])
    assert call(q=None) == tb.TB_EINVAL and call(c=None) == tb.TB_EINVAL
    for bad in (dict(base=None), dict(row=9217), dict(head=-256), dict(n=0), dict(n=15), dict(dtype=3), dict(dtype=tb.TB_F16), dict(base=A[4])):
        assert call(q=heads(**{"base": A[0], **bad})) == tb.TB_EINVAL, bad
    assert call(q=heads(A[0] + 8)) == tb.TB_EALIGN
    for bad in (dict(base=None), dict(n=8), dict(row=-8), dict(dtype=-1), dict(base=A[4])):
        assert call(gate=heads(**{"base": A[7], **bad})) == tb.TB_EINVAL, bad
    for bad in (dict(pages=0), dict(kv=0), dict(kv=3), dict(page=8), dict(dim=0), dict(dtype=tb.TB_F32), dict(k=None), dict(v=A[4]), dict(k=A[5])):
        assert call(c=cache(**bad)) == tb.TB_EINVAL, bad
    for dim in (16, 32, 96, 192, 512):
        assert call(c=cache(dim=dim)) == tb.TB_EUNSUPPORTED, dim
    c = cache()
    need = L.tb_attn_paged_workspace_bytes(ctypes.byref(c), 16, tb.TB_BF16, 3, 40)
    assert 0 < need <= 1 << 28
    assert call(ws_bytes=need - 1) == tb.TB_EINVAL
    for args in ((None, 16, 1, 3, 40), (cache(dim=96), 16, 1, 3, 40), (cache(), 15, 1, 3, 40), (cache(), 16, 2, 3, 40), (cache(), 16, 1, 0, 40),
                 (cache(), 16, 1, 3, 0), (cache(), 16, 1, 65537, 40), (cache(), 16, 1, 3, 1 << 27)):
        assert L.tb_attn_paged_workspace_bytes(ref(args[0]), *args[1:]) == 0


def test_attention_limits(L):
    """Sizes up to the last that an int holds are refused, not counted in 32 bits."""
    call = attn_call(L)
    far = dict(zip(ATTN, [(i + 2) << 54 for i in range(5)]))
    q = heads(1 << 54)
    c = cache(k=8 << 54, v=9 << 54)
    for sizes in (dict(requests=65537), dict(tokens=1 << 26), dict(tokens=LAST), dict(width=(1 << 26) + 1), dict(width=LAST), dict(requests=LAST),
                  dict(tokens=1 << 24, width=1 << 20), dict(requests=65536, width=1 << 20)):
        assert call(q=q, c=c, **far, **sizes) == tb.TB_EUNSUPPORTED, sizes


# ---- frequencies, and the tests' own plain implementations ---------------------------------
def test_frequencies():
    f, factor = tb.Rope.frequencies(64, 10000.0)
    assert factor == 1.0 and f.dtype.itemsize == 8
    assert np.allclose(f.numpy(), [10000.0 ** (-2 * i / 64) for i in range(32)], rtol=1e-14)
    g, factor = tb.Rope.frequencies(64, 10000.0, "linear", 4.0)
    assert factor == 1.0 and np.allclose(g.numpy(), f.numpy() / 4, rtol=1e-14)
    g, factor = tb.Rope.frequencies(64, 10000.0, "base", 4.0)
    assert factor == 1.0 and g[0] == f[0] and math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)
    g, factor = tb.Rope.frequencies(64, 10000.0, "parts", 4.0, trained=4096)
    turns = 4096 * f.numpy() / (2 * math.pi)
    assert math.isclose(factor, 0.1 * math.log(4) + 1)
    assert np.array_equal(g.numpy()[turns >= 32], f.numpy()[turns >= 32]) and (turns >= 32).any()
    assert np.allclose(g.numpy()[turns <= 1], f.numpy()[turns <= 1] / 4, rtol=1e-14) and (turns <= 1).any()
    between = (turns > 1) & (turns < 32)
    assert between.any() and (g.numpy()[between] < f.numpy()[between]).all() and (g.numpy()[between] > f.numpy()[between] / 4).all()
    for bad in ((0,), (63,), (64, -1.0), (64, 1e4, "other"), (64, 1e4, "parts", 4.0), (64, 1e4, "linear", 0.0)):
        with pytest.raises(tb.TbError):
            tb.Rope.frequencies(*bad)


def test_plain_plan():
    table = np.full((3, 4), -1, np.int32)
    table[0, :2], table[1, :1] = (5, 3), (7,)
    got = plain_kv.plan([20, 16, 0], [-1, 17, 1], 18, 16, 8, table, np.array([1, 2, 0]), 2)
    assert got["stack"] == [1] and got["left"] == 1               # 1 2 5 3 -> pops 3, 5, 2
    assert got["table"][1].tolist() == [7, 3, 5, -1] and got["table"][2].tolist() == [2, -1, -1, -1]
    assert got["lengths"] == [0, 33, 1] and got["offsets"] == [0, 0, 17, 18]
    assert got["slots"] == [48 + i for i in range(16)] + [80, 32] and got["missing"] == 0


def test_plain_attention():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal(s) for s in ((2, 2, 8), (3, 1, 16, 8), (3, 1, 16, 8)))
    table = np.array([[2, 0]])
    out, size, big, keys = plain_kv.attention(q, k, v, table, [0, 2], [20], 0.5)
    kk, vv = (np.concatenate([x[2, 0], x[0, 0]]) for x in (k, v))
    for i in range(2):
        for h in range(2):
            w = np.exp(kk[:19 + i] @ q[i, h] * 0.5)
            assert np.allclose(out[i, h], w @ vv[:19 + i] / w.sum()) and keys[i, h] == 19 + i
    x, size = plain_kv.rope(q, np.array([3, 4]), np.array([0.1, 0.2]), 1.0, True)
    assert np.allclose(x[0, 0, 0], q[0, 0, 0] * math.cos(0.3) - q[0, 0, 1] * math.sin(0.3))
    assert np.allclose(x[1, 1, 3], q[1, 1, 3] * math.cos(0.8) + q[1, 1, 2] * math.sin(0.8)) and np.array_equal(x[..., 4:], q[..., 4:])
    x, size = plain_kv.rope(q, np.array([3, 4]), np.array([0.1, 0.2]), 2.0, False)
    assert np.allclose(x[0, 0, 1], 2 * (q[0, 0, 1] * math.cos(0.6) - q[0, 0, 3] * math.sin(0.6)))
