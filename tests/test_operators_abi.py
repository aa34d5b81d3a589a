"""Refusals of the row, 4-bit and expert operators, without a GPU: no call here reaches a launch."""

import ctypes
import os

import numpy as np
import pytest

import ternary_weight_int8_tb_amd as tb
from tests import plain
from ternary_weight_int8_tb_amd import build as tb_build

A = [0x10000000 * (i + 1) for i in range(14)]      # fake 16-byte aligned addresses, 256 MiB apart


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(tb.LIB_PATH):
        tb_build.build()
    return tb.lib()


def refused(call, args, name, value, status=tb.TB_EINVAL):
    got = call(**{**args, name: value})
    assert got == status, (name, value, got)


def common(call, arrays, sizes=()):
    """Null, misaligned and overlapping arrays. arrays: name -> (address, is an output)."""
    args = {n: a for n, (a, _) in arrays.items()}
    for n, (a, out) in arrays.items():
        refused(call, args, n, None)
        refused(call, args, n, a + 4, tb.TB_EALIGN)
        for n2, (a2, out2) in arrays.items():
            if n != n2 and (out or out2):
                refused(call, args, n, a2 + 16)
    for n, values in sizes:
        for v in values:
            refused(call, args, n, v)


def test_norm(L):
    def call(x=A[0], res=A[1], gamma=A[2], dtype=1, m=2, k=512, eps=1e-6, res_out=A[3], y=A[4], q=A[5], dq=A[6]):
        return L.tb_add_rmsnorm_quant_i8(x, res, gamma, dtype, m, k, eps, res_out, y, q, dq, None)
    for n in ("x", "gamma", "q", "dq"):
        assert call(**{n: None}) == tb.TB_EINVAL, n
    for i, n in enumerate(("x", "res", "gamma", "res_out", "y", "q", "dq")):
        assert call(**{n: A[i] + 8}) == tb.TB_EALIGN, n
    outs, ins = ("y", "q", "dq"), ("x", "res", "gamma", "res_out")
    addr = dict(zip(("x", "res", "gamma", "res_out", "y", "q", "dq"), A))
    for o in outs:
        for other in addr:
            if o != other:
                assert call(**{o: addr[other] + 16}) == tb.TB_EINVAL, (o, other)
    assert call(res_out=A[0] + 64) == tb.TB_EINVAL          # neither x itself nor apart from it
    assert call(res_out=A[1] + 64) == tb.TB_EINVAL
    assert call(res=A[0] + 64, res_out=A[0]) == tb.TB_EINVAL  # in place, and the other input overlaps
    assert call(gamma=A[0], res_out=A[0]) == tb.TB_EINVAL
    for n, values in (("dtype", (-1, 3)), ("m", (0, -1)), ("k", (0, 64, 500, -128)), ("eps", (-1e-6, float("nan"), float("inf")))):
        for v in values:
            assert call(**{n: v}) == tb.TB_EINVAL, (n, v)
    assert call(k=128 * 15361, m=1, x=1 << 40, res=None, res_out=None, y=None, gamma=2 << 40, q=3 << 40, dq=4 << 40) == tb.TB_EUNSUPPORTED


def test_mx_quant_and_dequant(L):
    def quant(x=A[0], dtype=1, m=2, k=512, rotate=0, codes=A[1], scales=A[2]):
        return L.tb_mxfp4_quant(x, dtype, m, k, rotate, codes, scales, None)

    def dequant(codes=A[0], scales=A[1], m=2, k=512, y=A[2], dtype=0):
        return L.tb_mxfp4_dequant(codes, scales, m, k, y, dtype, None)
    sizes = [("dtype", (-1, 3)), ("m", (0, -5)), ("k", (0, 32, 96, 100, -128))]
    common(quant, {"x": (A[0], False), "codes": (A[1], True), "scales": (A[2], True)}, sizes + [("rotate", (2, -1))])
    common(dequant, {"codes": (A[0], False), "scales": (A[1], False), "y": (A[2], True)}, sizes)


def test_mx_gemm(L):
    def call(wcodes=A[0], wscales=A[1], n=64, k=512, codes=A[2], scales=A[3], m=2, y=A[4], dtype=0, ws=A[5], ws_bytes=1 << 27):
        w = tb.CMxfp4(wcodes, wscales, n, k)
        return L.tb_mxfp4_gemm(ctypes.byref(w), codes, scales, m, y, dtype, ws, ws_bytes, None)
    common(call, {"wcodes": (A[0], False), "wscales": (A[1], False), "codes": (A[2], False), "scales": (A[3], False), "y": (A[4], True)},
           [("n", (0, -1)), ("k", (0, 64, 500)), ("m", (0, -1)), ("dtype", (-1, 3))])
    assert L.tb_mxfp4_gemm(None, A[2], A[3], 1, A[4], 0, A[5], 1 << 27, None) == tb.TB_EINVAL
    # a shape that needs a workspace refuses one that is missing, too small or misaligned
    for m, n, k in ((128, 512, 17408), (256, 1024, 8192), (96, 640, 17408)):
        w = tb.CMxfp4(A[0], A[1], n, k)
        need = L.tb_mxfp4_gemm_workspace_bytes(ctypes.byref(w), m)
        if need:
            args = dict(n=n, k=k, m=m)
            assert call(**args, ws=None) == tb.TB_EINVAL
            assert call(**args, ws_bytes=need - 1) == tb.TB_EINVAL
            assert call(**args, ws=A[5] + 8) == tb.TB_EALIGN
            assert call(**args, ws=A[4]) == tb.TB_EINVAL
    bad = tb.CMxfp4(A[0], A[1], 0, 512)
    assert L.tb_mxfp4_gemm_workspace_bytes(ctypes.byref(bad), 4) == 0
    assert L.tb_mxfp4_gemm_workspace_bytes(None, 4) == 0


def experts(base, e=4, n=256, k=512, fmt=0):
    return tb.CExperts(A[base], A[base + 1], e, n, k, fmt)


def test_moe_plan(L):
    def call(ids=A[0], tokens=8, topk=2, experts=4, offsets=A[1], order=A[2]):
        return L.tb_moe_plan(ids, tokens, topk, experts, offsets, order, None)
    common(call, {"ids": (A[0], False), "offsets": (A[1], True), "order": (A[2], True)},
           [("tokens", (0, -1)), ("topk", (0, -3)), ("experts", (0, -1))])
    assert call(experts=65537) == tb.TB_EUNSUPPORTED
    assert call(tokens=1 << 30, topk=2) == tb.TB_EUNSUPPORTED


def test_moe_products(L):
    names = ("q", "dq", "offsets", "order", "h", "qh", "dqh")

    def gateup(wg=None, wu=None, tokens=8, topk=2, **a):
        a = {**dict(zip(names, A[4:11])), **a}
        wg, wu = wg or experts(0), wu or experts(2)
        return L.tb_moe_gateup_silu(ctypes.byref(wg), ctypes.byref(wu), a["q"], a["dq"], tokens, topk, a["offsets"], a["order"],
                                    a["h"], a["qh"], a["dqh"], None)

    def down(wd=None, pairs=16, **a):
        a = {**dict(zip(("qh", "dqh", "offsets", "order", "y"), A[2:7])), **a}
        wd = wd or experts(0)
        return L.tb_moe_down(ctypes.byref(wd), a["qh"], a["dqh"], pairs, a["offsets"], a["order"], a["y"], None)
    common(lambda **a: gateup(**a), {n: (v, n in ("h", "qh", "dqh")) for n, v in zip(names, A[4:11])},
           [("tokens", (0, -1)), ("topk", (0,))])
    common(lambda **a: down(**a), {n: (v, n == "y") for n, v in zip(("qh", "dqh", "offsets", "order", "y"), A[2:7])},
           [("pairs", (0, -1))])
    for n in ("h", "qh", "dqh"):
        assert gateup(**{n: A[0] + 64}) == tb.TB_EINVAL          # an output over the codes
    for bad in (dict(e=0), dict(n=0), dict(k=0), dict(k=500), dict(fmt=3), dict(fmt=-1), dict(e=5), dict(n=128), dict(k=256), dict(fmt=1)):
        assert gateup(wu=experts(2, **bad)) == tb.TB_EINVAL, bad
    for bad in (dict(e=0), dict(n=0), dict(k=64), dict(fmt=7)):
        assert down(wd=experts(0, **bad)) == tb.TB_EINVAL, bad
    odd = dict(n=200)                                            # h is rotated in blocks of 128
    assert gateup(wg=experts(0, **odd), wu=experts(2, **odd)) == tb.TB_EINVAL
    ri4 = dict(fmt=tb.TB_FMT_SIGN1_RI4)
    assert gateup(wg=experts(0, **ri4), wu=experts(2, **ri4)) == tb.TB_EUNSUPPORTED
    assert down(wd=experts(0, **ri4)) == tb.TB_EUNSUPPORTED
    assert down(wd=tb.CExperts(A[0] + 2, A[1], 4, 256, 512, 0)) == tb.TB_EALIGN
    assert down(wd=tb.CExperts(None, A[1], 4, 256, 512, 0)) == tb.TB_EINVAL
    assert down(wd=experts(0, e=65537, n=1, k=128)) == tb.TB_EUNSUPPORTED
    assert L.tb_moe_down(None, A[2], A[3], 4, A[4], A[5], A[6], None) == tb.TB_EINVAL


def test_moe_combine(L):
    def call(y=A[0], weights=A[1], ids=A[2], tokens=8, topk=2, experts=4, n=256, out=A[3], dtype=1):
        return L.tb_moe_combine(y, weights, ids, tokens, topk, experts, n, out, dtype, None)
    common(call, {"y": (A[0], False), "weights": (A[1], False), "ids": (A[2], False), "out": (A[3], True)},
           [("tokens", (0, -1)), ("topk", (0,)), ("experts", (0,)), ("n", (0, -1)), ("dtype", (3, -1))])
    assert call(tokens=1 << 30, topk=4) == tb.TB_EUNSUPPORTED


def test_mx_gemm_limits(L):
    """Sizes up to the last that an int holds are refused, not counted in 32 bits."""
    last = 2 ** 31 - 1
    far = [(i + 1) << 52 for i in range(6)]   # apart, whatever the sizes

    def call(m, n, k):
        w = tb.CMxfp4(far[0], far[1], n, k)
        assert L.tb_mxfp4_gemm_workspace_bytes(ctypes.byref(w), m) == 0
        return L.tb_mxfp4_gemm(ctypes.byref(w), far[2], far[3], m, far[4], 1, far[5], 2 ** 63, None)
    for m in (last, last - 100, last - 127):
        assert call(m, 16, 128) == tb.TB_EUNSUPPORTED, m
        assert call(16, m, 128) == tb.TB_EUNSUPPORTED, m
    assert call(last, last, 128) == tb.TB_EUNSUPPORTED
    assert call((1 << 30) + 1, 1, 128) == tb.TB_EUNSUPPORTED   # past 2^23 tiles of 128 x 128
    assert call(1, 1, 1 << 24) == tb.TB_EUNSUPPORTED
    assert call(1 << 20, 1 << 20, 128) == tb.TB_EUNSUPPORTED


def test_moe_combine_limits(L):
    """Columns are counted in 31 bits: the last workgroup's have to fit too."""
    far = [(i + 1) << 52 for i in range(4)]
    for n in (2 ** 31 - 1, 2 ** 31 - 4, 2 ** 31 - 1023):
        assert L.tb_moe_combine(far[0], far[1], far[2], 1, 1, 4, n, far[3], 1, None) == tb.TB_EUNSUPPORTED, n


# ---- the tests' own plain implementations -----------------------------------------------
def test_plain_transform_and_formats():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 256)).astype(np.float32)
    exact = (x.astype(np.float64).reshape(-1, 128) @ plain.hadamard()).reshape(3, 256)
    assert np.abs(plain.wht32(x) - exact).max() < 1e-4
    every = np.tile(np.concatenate([plain.LEVELS, -plain.LEVELS]), 16).astype(np.float32)[None]
    codes, scales = plain.mx_quant(every)
    assert (scales == 127).all() and np.array_equal(plain.mx_values(codes, scales), every)
    codes, scales = plain.mx_quant(x)
    v = plain.mx_values(codes, scales)
    # half a step: at most 1/4 of the scale below 2, 1 above 4; values of 6 to 8 saturate
    step = 2.0 ** (scales.astype(np.float64) - 127).repeat(32, axis=1)
    assert np.all(np.abs(v - x) <= np.where(np.abs(x) > 6 * step, 2.0, 1.0) * step)
