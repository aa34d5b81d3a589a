"""Residual + RMSNorm + rotated int8 rows on MI355X, against the definition.

The stored residual and the codes are exact (the definition fixes every rounding up to them); the
scales and the normed rows carry the rounding of one factor per row.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import ternary_weight_int8_tb_amd as tb
from tests import gpu_util as gu
from tests import plain
from tests.plain import U

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def rows(m, k, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.where(torch.rand(k, generator=g) < 0.02, 20.0, 1.0)
    return x.to(dtype).to(gu.DEV)


class Out:
    def __init__(self, m, k, dtype):
        nan = float("nan")
        self.s = torch.full((m, k), nan, dtype=dtype, device=gu.DEV)
        self.y = torch.full((m, k), nan, dtype=dtype, device=gu.DEV)
        self.q, self.dq = gu.i8_out(m, k), gu.f32_out(m, k // 128)


def check(x, res, gamma, eps, s, y, q, dq):
    """s, q exact; dq and y within their roundings. (s or y may be None.)"""
    m, k = x.shape
    total = x.cpu().float() + res.cpu().float() if res is not None else x.cpu().float()
    want_s = total.to(x.dtype)
    if s is not None:
        assert torch.equal(s.cpu(), want_s)
    s32 = want_s.float().numpy()
    g = gamma.cpu().numpy()
    codes, amax = plain.quant_i8(plain.wht32(s32 * g))
    assert np.array_equal(gu.host(q), codes)
    s64 = s32.astype(np.float64)
    f = 1.0 / np.sqrt((s64 * s64).mean(-1, keepdims=True) + eps)
    # f: squares of 8 elements summed in fp32 (8 roundings, halved by the root) and one rounding;
    # then f * unit, amax * that, and unit itself: 4 + 1 + 3 half steps
    want = amax.astype(np.float64) * f / (127 * np.sqrt(128.0))
    got = gu.host(dq).astype(np.float64)
    assert np.all(np.abs(got - want) <= 8.01 * U * np.abs(want))
    if y is not None:
        # 5 half steps of f, the two products, and the type's own rounding
        want = s64 * f * g
        tiny = {torch.float16: 2.0 ** -25}.get(y.dtype, 0.0)   # half a step of an fp16 subnormal
        tol = (7.01 * U + torch.finfo(y.dtype).eps / 2) * np.abs(want) + tiny
        assert np.all(np.abs(f64(y) - want) <= tol)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", [128, 256, 384, 5120, 8192, 8320, 17408])
@pytest.mark.parametrize("m", [1, 2, 37])
def test_norm(m, k, dtype):
    print(f"norm m={m} k={k} {dtype}", flush=True)
    dt = TYPES[dtype]
    x, res = rows(m, k, dt, 1), rows(m, k, dt, 2)
    gamma = 1 + 0.3 * torch.randn(k, device=gu.DEV)
    o = Out(m, k, dt)
    tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-6, o.s, o.y, o.q, o.dq)
    check(x, res, gamma, 1e-6, o.s, o.y, o.q, o.dq)


# more rows than workgroups are launched, in one to four passes over a row
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,k", [(8300, 128), (5500, 1280), (1100, 8192), (1100, 8320), (600, 17408), (700, 24704)])
def test_norm_many_rows(m, k, dtype):
    print(f"norm m={m} k={k} {dtype}", flush=True)
    dt = TYPES[dtype]
    x, res = rows(m, k, dt, 11), rows(m, k, dt, 12)
    gamma = 1 + 0.3 * torch.randn(k, device=gu.DEV)
    o = Out(m, k, dt)
    tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-6, o.s, o.y, o.q, o.dq)
    check(x, res, gamma, 1e-6, o.s, o.y, o.q, o.dq)
    # in place, without y: the same codes
    q, dq = o.q.clone(), o.dq.clone()
    tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-6, res, None, o.q, o.dq)
    assert torch.equal(o.q, q) and torch.equal(o.dq, dq) and torch.equal(res, o.s)


@pytest.mark.parametrize("has_res,has_out,has_y", [(r, o, y) for r in (0, 1) for o in (0, 1) for y in (0, 1)])
def test_norm_optional_arrays(has_res, has_out, has_y):
    m, k = 5, 1280
    x = rows(m, k, torch.bfloat16, 3)
    res = rows(m, k, torch.bfloat16, 4) if has_res else None
    gamma = 1 + 0.3 * torch.randn(k, device=gu.DEV)
    o = Out(m, k, torch.bfloat16)
    tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-5, o.s if has_out else None, o.y if has_y else None, o.q, o.dq)
    check(x, res, gamma, 1e-5, o.s if has_out else None, o.y if has_y else None, o.q, o.dq)


@pytest.mark.parametrize("place", ["x", "res", "both"])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_in_place(place, dtype):
    m, k = 7, 8320
    x, res = rows(m, k, TYPES[dtype], 5), rows(m, k, TYPES[dtype], 6)
    gamma = 1 + 0.3 * torch.randn(k, device=gu.DEV)
    if place == "both":   # x + x, into x
        res = x
    x0, res0 = x.clone(), res.clone()
    o = Out(m, k, TYPES[dtype])
    target = res if place == "res" else x
    tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-6, target, o.y, o.q, o.dq)
    check(x0, res0, gamma, 1e-6, target, o.y, o.q, o.dq)


def test_norm_zero_and_tiny_rows():
    k = 512
    x = torch.zeros(5, k, device=gu.DEV)
    x[1, :128] = torch.randn(128, device=gu.DEV)          # the other blocks are zero
    x[2] = torch.randn(k, device=gu.DEV) * 1e-34          # below 2^-100: counts as zero
    x[3] = torch.randn(k, device=gu.DEV) * 1e17           # squares sum to 1e36
    x[4, 5] = 1.0
    gamma = torch.ones(k, device=gu.DEV)
    o = Out(5, k, torch.float32)
    tb.tb_add_rmsnorm_quant_i8(x, None, gamma, 1e-6, o.s, o.y, o.q, o.dq)
    check(x, None, gamma, 1e-6, o.s, None, o.q, o.dq)
    q, dq = gu.host(o.q), gu.host(o.dq)
    assert not q[0].any() and not dq[0].any() and not q[1, 128:].any() and not q[2].any() and not dq[2].any()
    tb.tb_add_rmsnorm_quant_i8(x, None, gamma, 0.0, o.s, o.y, o.q, o.dq)
    assert not gu.host(o.y)[0].any() and not gu.host(o.dq)[0].any()


@pytest.mark.parametrize("k", [512, 8320])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_rows_that_are_not_finite(k, dtype):
    m, dt = 6, TYPES[dtype]
    x, gamma = rows(m, k, dt, 21), 1 + 0.3 * torch.randn(k, device=gu.DEV)
    clean = Out(m, k, dt)
    tb.tb_add_rmsnorm_quant_i8(x, None, gamma, 1e-6, None, clean.y, clean.q, clean.dq)
    x[1, 130], x[3, 5], x[4, k - 1] = float("nan"), float("inf"), float("-inf")
    o = Out(m, k, dt)
    tb.tb_add_rmsnorm_quant_i8(x, None, gamma, 1e-6, None, o.y, o.q, o.dq)
    good = [0, 2, 5]
    for a, b in ((o.q, clean.q), (o.dq, clean.dq), (o.y, clean.y)):
        assert torch.equal(a[good], b[good])
    assert torch.isnan(o.dq[1]).all() and torch.isnan(o.y[1]).all()
    for row, block in ((1, 1), (3, 0), (4, k // 128 - 1)):
        assert torch.isnan(o.dq[row, block]) and not o.q[row, 128 * block:128 * (block + 1)].any()
    for row, block in ((3, 0), (4, k // 128 - 1)):   # the mean is infinite: f = 0
        others = [b for b in range(k // 128) if b != block]
        assert not o.dq[row, others].any()


def test_norm_large_offsets():
    """Rows past 4 GiB have the bits that they have alone."""
    m, k = 270003, 8192
    x = torch.empty(m, k, dtype=torch.bfloat16, device=gu.DEV).normal_()
    gamma = 1 + 0.3 * torch.randn(k, device=gu.DEV)
    s, q, dq = torch.empty_like(x), gu.i8_out(m, k), gu.f32_out(m, k // 128)
    tb.tb_add_rmsnorm_quant_i8(x, x, gamma, 1e-6, s, None, q, dq)
    codes = torch.empty(m, k // 2, dtype=torch.uint8, device=gu.DEV)
    scales = torch.empty(m, k // 32, dtype=torch.uint8, device=gu.DEV)
    tb.tb_mxfp4_quant(s, codes, scales, True)
    for a in (0, 131071, m - 3):
        part = x[a:a + 3].clone()
        s2, q2, dq2 = torch.empty_like(part), gu.i8_out(3, k), gu.f32_out(3, k // 128)
        tb.tb_add_rmsnorm_quant_i8(part, part, gamma, 1e-6, s2, None, q2, dq2)
        c2, sc2 = torch.empty_like(codes[:3]), torch.empty_like(scales[:3])
        tb.tb_mxfp4_quant(s2, c2, sc2, True)
        for all_rows, alone in ((s, s2), (q, q2), (dq, dq2), (codes, c2), (scales, sc2)):
            assert torch.equal(all_rows[a:a + 3], alone)


def test_norm_codes_are_those_of_the_quantiser():
    # gamma = 1, no residual: the codes of tb_rotate_quant_i8 on the same rows
    x = rows(8, 5120, torch.float32, 7)
    o = Out(8, 5120, torch.float32)
    tb.tb_add_rmsnorm_quant_i8(x, None, torch.ones(5120, device=gu.DEV), 1e-6, None, None, o.q, o.dq)
    q, dq = gu.i8_out(8, 5120), gu.f32_out(8, 40)
    tb.tb_rotate_quant_i8(x, q, dq)
    assert torch.equal(o.q, q)
    qo, _ = oracle.default().rotate_quant(x.cpu().numpy())
    assert np.array_equal(gu.host(o.q), qo)


def test_norm_rows_do_not_depend_on_each_other():
    x, res = rows(300, 2560, torch.bfloat16, 8), rows(300, 2560, torch.bfloat16, 9)
    gamma = 1 + 0.3 * torch.randn(2560, device=gu.DEV)
    o, one = Out(300, 2560, torch.bfloat16), Out(1, 2560, torch.bfloat16)
    tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-6, o.s, o.y, o.q, o.dq)
    for r in (0, 17, 299):
        tb.tb_add_rmsnorm_quant_i8(x[r:r + 1], res[r:r + 1], gamma, 1e-6, one.s, one.y, one.q, one.dq)
        for name in ("s", "y", "q", "dq"):
            assert torch.equal(getattr(o, name)[r:r + 1], getattr(one, name)), name


def test_norm_graph_and_stream():
    m, k = 24, 5120
    x, res = rows(m, k, torch.bfloat16, 10), rows(m, k, torch.bfloat16, 11)
    gamma = 1 + 0.3 * torch.randn(k, device=gu.DEV)
    o = Out(m, k, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-6, o.s, o.y, o.q, o.dq, stream=side)
    torch.cuda.synchronize()
    check(x, res, gamma, 1e-6, o.s, o.y, o.q, o.dq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-6, o.s, o.y, o.q, o.dq)
    for r in range(3):
        x.copy_(rows(m, k, torch.bfloat16, 20 + r))
        o.q.fill_(0x5A), o.dq.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(x, res, gamma, 1e-6, o.s, o.y, o.q, o.dq)


def test_norm_then_product():
    # the rows go straight into a product of the library
    from ternary_weight_int8_tb_amd import synth
    w = synth.matrix(synth.FMT_TERNARY2, 640, 1280, 90, 0, synth.T_DOWN)
    x, res = rows(4, 1280, torch.bfloat16, 12), rows(4, 1280, torch.bfloat16, 13)
    gamma = 1 + 0.3 * torch.randn(1280, device=gu.DEV)
    o = Out(4, 1280, torch.bfloat16)
    tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-6, o.s, None, o.q, o.dq)
    y = gu.f32_out(4, 640)
    tb.tb_gemv_ternary(tb.Matrix.upload(w), o.q, o.dq, y)
    ref, sabs = oracle.default().gemv(w, gu.host(o.q), gu.host(o.dq))
    assert np.all(np.abs(gu.host(y) - ref) <= 1e-4 * sabs + 1e-30)


def test_norm_binding_refusals():
    x = rows(4, 256, torch.bfloat16, 14)
    gamma, o = torch.ones(256, device=gu.DEV), Out(4, 256, torch.bfloat16)

    def call(x=x, res=None, gamma=gamma, res_out=None, y=None, q=o.q, dq=o.dq):
        with pytest.raises(tb.TbError):
            tb.tb_add_rmsnorm_quant_i8(x, res, gamma, 1e-6, res_out, y, q, dq)
    call(x=x.double())
    call(x=x.cpu())
    call(x=x.t())
    call(x=x[0])
    call(res=x.float())
    call(res=rows(3, 256, torch.bfloat16, 1))
    call(res=rows(4, 512, torch.bfloat16, 1)[:, ::2])
    call(gamma=gamma.bfloat16())
    call(gamma=gamma.cpu())
    call(res_out=o.s.float())
    call(y=o.y[:3])
    call(q=o.q.to(torch.uint8))
    call(dq=o.dq[:, :1])
    call(y=x)                      # y may not be an input
    assert (gu.host(o.q) == gu.POISON_I8).all()


@pytest.mark.parametrize("k", [512, 8320])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_zero_block_of_a_row_with_a_nan(k, dtype):
    x = rows(3, k, TYPES[dtype], 30)
    x[1:, :128] = 0
    x[1, k - 1] = float("nan")
    o = Out(3, k, TYPES[dtype])
    tb.tb_add_rmsnorm_quant_i8(x, None, torch.ones(k, device=gu.DEV), 1e-6, None, o.y, o.q, o.dq)
    assert torch.isnan(o.dq[1]).all() and torch.isnan(o.y[1]).all() and not o.q[1, :128].any()
    assert o.dq[2, 0] == 0 and (o.dq[2, 1:] > 0).all()   # without a NaN it stays a block of zeros


@pytest.mark.parametrize("k", [512, 8320])
def test_norm_block_whose_rotation_overflows(k):
    """Finite rows, u past the largest fp32: with infinities alone, and with NaN among them."""
    x = rows(3, k, torch.float32, 31)
    x[:2, :128] = 0
    x[0, :4] = 1          # 4 x 1e38 is infinite, and nothing is subtracted from it
    x[1, :8] = 1
    gamma = torch.ones(k, device=gu.DEV)
    gamma[:128] = 1e38
    x[2, :128] = 0
    o = Out(3, k, torch.float32)
    tb.tb_add_rmsnorm_quant_i8(x, None, gamma, 1e-6, None, o.y, o.q, o.dq)
    assert torch.isnan(o.dq[:2, 0]).all() and not o.q[:, :128].any() and o.dq[2, 0] == 0
    assert torch.isfinite(o.dq[:, 1:]).all() and torch.isfinite(o.y).all()


@pytest.mark.parametrize("k", [512, 8320])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("power", [-120, -90, -70, 58, 70, 90, 110])
def test_norm_rows_of_any_size(k, dtype, power):
    """Squares that fp32 cannot hold, eps = 0."""
    x = (rows(4, k, torch.float32, 32) * 2.0 ** power).to(TYPES[dtype])
    x[3] = 0
    gamma = 1 + 0.3 * torch.randn(k, device=gu.DEV)
    o = Out(4, k, TYPES[dtype])
    tb.tb_add_rmsnorm_quant_i8(x, None, gamma, 0.0, o.s, o.y, o.q, o.dq)
    check(x[:3], None, gamma, 0.0, o.s[:3], o.y[:3], o.q[:3], o.dq[:3])
    assert not o.y[3].any() and not o.q[3].any() and not o.dq[3].any()


def test_norm_largest_and_smallest_rows():
    k = 512
    x = torch.zeros(3, k, device=gu.DEV)
    x[0, 7] = 3e38
    x[1, 300] = -1e-38
    x[2] = 2.0 ** -148       # f is past the largest fp32
    gamma = 1 + 0.3 * torch.randn(k, device=gu.DEV)
    o = Out(3, k, torch.float32)
    tb.tb_add_rmsnorm_quant_i8(x, None, gamma, 0.0, o.s, o.y, o.q, o.dq)
    # one element: its normed value is sqrt(k); equal ones: 1. f has 24 bits whatever its exponent: a rounding of f,
    # two of the products, and one to spare
    g = gamma.double().cpu().numpy()
    y = f64(o.y)
    for row, col, want in ((0, 7, np.sqrt(k) * g[7]), (1, 300, -np.sqrt(k) * g[300])):
        assert abs(y[row, col] - want) <= 4 * U * abs(want)
        assert not np.delete(y[row], col).any()
    assert np.all(np.abs(y[2] - g) <= 4 * U * np.abs(g))


@pytest.mark.parametrize("k", [512, 8320])
def test_norm_scales_of_the_largest_and_smallest_rows(k):
    x, gamma = torch.zeros(2, k, device=gu.DEV), torch.ones(k, device=gu.DEV)
    x[0, 7] = 3e38
    x[1, 300] = 2.0 ** -140
    gamma[300] = 2.0 ** 100   # the block's amax is 2^-40
    o = Out(2, k, torch.float32)
    tb.tb_add_rmsnorm_quant_i8(x, None, gamma, 0.0, None, o.y, o.q, o.dq)
    # roundings of f, of unit, of their product and of amax times it, and one to spare
    for row, block, g in ((0, 0, 1.0), (1, 2, 2.0 ** 100)):
        want = g * np.sqrt(k) / (127 * np.sqrt(128.0))
        assert abs(float(o.dq[row, block]) - want) <= 5 * U * want
        assert not np.delete(gu.host(o.dq)[row], block).any()
        assert (np.abs(gu.host(o.q)[row, 128 * block:128 * (block + 1)]) == 127).all()
