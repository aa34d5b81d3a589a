"""Microscaled 4-bit rows and their product on MI355X, against plain implementations in 64 bits."""

from __future__ import annotations

import numpy as np
import pytest
import torch

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


def u8_out(*shape):
    return torch.full(shape, 0xA5, dtype=torch.uint8, device=gu.DEV)


def quant(x, rotate=False):
    m, k = x.shape
    codes, scales = u8_out(m, k // 2), u8_out(m, k // 32)
    tb.tb_mxfp4_quant(x, codes, scales, rotate)
    return codes, scales


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,k", [(1, 128), (3, 384), (5, 5120), (129, 640)])
@pytest.mark.parametrize("rotate", [False, True])
def test_quant(m, k, dtype, rotate):
    print(f"mx quant m={m} k={k} {dtype} rotate={rotate}", flush=True)
    g = torch.Generator().manual_seed(m * k)
    x = (torch.randn(m, k, generator=g) * torch.exp2(torch.randint(-12, 13, (m, k // 32, 1), generator=g).float())
         .expand(m, k // 32, 32).reshape(m, k)).to(TYPES[dtype])
    x32 = x.float().numpy()
    if rotate:
        x32 = plain.wht32(x32) * np.float32(1 / np.sqrt(128.0))
    codes, scales = quant(x.to(gu.DEV), rotate)
    want_c, want_s = plain.mx_quant(x32)
    assert np.array_equal(gu.host(scales), want_s)
    assert np.array_equal(gu.host(codes), want_c)


def test_quant_borders():
    """Every border between two values, one fp32 step below and above it, at several exponents."""
    mids = (plain.LEVELS[1:] + plain.LEVELS[:-1]) / 2
    vals = np.concatenate([[m, np.nextafter(np.float32(m), np.float32(0)), np.nextafter(np.float32(m), np.float32(9))]
                           for m in mids] + [plain.LEVELS, [7.0, 7.5, 7.99]]).astype(np.float32)
    vals = np.concatenate([vals, -vals])
    rows = []
    for e in (-120, -60, -3, 0, 5, 100, 125):
        for i in range(0, len(vals), 31):
            b = np.zeros(32, np.float32)
            b[:len(vals[i:i + 31])] = vals[i:i + 31]
            b[31] = 7.9        # fixes the scale at 2^e
            rows.append(b * np.float32(2.0) ** e)
    while len(rows) % 4:
        rows.append(np.zeros(32, np.float32))
    x = np.stack(rows).reshape(-1, 128)
    codes, scales = quant(torch.from_numpy(x).to(gu.DEV))
    want_c, want_s = plain.mx_quant(x)
    assert np.array_equal(gu.host(scales), want_s)
    assert np.array_equal(gu.host(codes), want_c)


def test_quant_zero_tiny_and_not_finite():
    x = np.random.default_rng(1).standard_normal((6, 128)).astype(np.float32)
    x[0] = 0
    x[1] *= 2.0 ** -130
    x[2, 5], x[2, 40], x[2, 70] = np.nan, np.inf, -np.inf
    x[3, :32] = 0
    x[4, :32] = -0.0
    x[5, :32] = np.float32(2.0 ** -124)      # the smallest block that is kept
    x[5, 32:64] = np.nextafter(np.float32(2.0 ** -124), np.float32(0))
    codes, scales = quant(torch.from_numpy(x).to(gu.DEV))
    want_c, want_s = plain.mx_quant(x)
    assert want_s[5, 0] == 1 and want_s[5, 1] == 0
    assert np.array_equal(gu.host(scales), want_s)
    assert np.array_equal(gu.host(codes), want_c)
    y = gu.f32_out(6, 128)
    tb.tb_mxfp4_dequant(codes, scales, y)
    assert np.array_equal(gu.host(y), plain.mx_values(want_c, want_s).astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_dequant(dtype):
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 256, (257, 128), dtype=np.uint8)
    scales = rng.integers(0, 256, (257, 8), dtype=np.uint8)
    y = torch.full((257, 256), float("nan"), dtype=TYPES[dtype], device=gu.DEV)
    tb.tb_mxfp4_dequant(gu.dev(codes), gu.dev(scales), y)
    want = torch.from_numpy(plain.mx_values(codes, scales)).to(torch.float32).to(TYPES[dtype])
    assert np.array_equal(y.float().cpu().numpy(), want.float().numpy(), equal_nan=True)


def gemm(ac, asc, wc, ws, dtype=torch.float32):
    w = tb.Mxfp4(gu.dev(wc), gu.dev(ws))
    m = ac.shape[0]
    need = tb.tb_mxfp4_gemm_workspace_bytes(w, m)
    work = u8_out(need) if need else None
    y = torch.full((m, w.n), float("nan"), dtype=dtype, device=gu.DEV)
    tb.tb_mxfp4_gemm(w, gu.dev(ac), gu.dev(asc), y, work)
    torch.cuda.synchronize()
    return y


def operands(m, n, k, seed, lo, hi):
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 256, (m, k // 2), dtype=np.uint8), rng.integers(lo, hi, (m, k // 32), dtype=np.uint8),
            rng.integers(0, 256, (n, k // 2), dtype=np.uint8), rng.integers(lo, hi, (n, k // 32), dtype=np.uint8))


SHAPES = [(1, 16, 128), (1, 1, 128), (1, 5120, 5120), (2, 17, 256), (15, 33, 384), (16, 64, 1280), (17, 100, 640), (31, 9, 2048),
          (33, 250, 896), (64, 128, 512), (65, 129, 256), (100, 77, 17408), (127, 300, 1152), (129, 513, 384), (200, 1000, 4096),
          (256, 256, 128), (257, 260, 256), (300, 511, 768), (513, 255, 5120), (640, 768, 2560), (1000, 1030, 1024)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_exact(m, n, k):
    """Scale 1 everywhere: all products are multiples of 1/4 and all sums stay below 2^24 / 4
    (36 * 17408 < 2^22), so fp32 holds every partial sum exactly, in any order."""
    print(f"mx gemm exact {m} {n} {k}", flush=True)
    ac, asc, wc, ws = operands(m, n, k, m + n + k, 127, 128)
    want = plain.mx_values(ac, asc) @ plain.mx_values(wc, ws).T
    assert np.array_equal(gu.host(gemm(ac, asc, wc, ws)), want.astype(np.float32))


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_gemm(m, n, k, dtype):
    """Scales over 7 binades. A sum of k terms in fp32, in any order and with sums cut instead of
    rounded, is within 2 k U sum|terms|; the output is rounded once."""
    print(f"mx gemm {m} {n} {k} {dtype}", flush=True)
    ac, asc, wc, ws = operands(m, n, k, m * n + k, 117, 124)
    a, w = plain.mx_values(ac, asc), plain.mx_values(wc, ws)
    want, size = a @ w.T, np.abs(a) @ np.abs(w).T
    y = gemm(ac, asc, wc, ws, TYPES[dtype])
    got = y.double().cpu().numpy()
    tol = 2 * k * U * size + torch.finfo(TYPES[dtype]).eps / 2 * np.abs(want) * (1 + 1e-3) + 2.0 ** -25 * (dtype == "f16")
    assert np.all(np.abs(got - want) <= tol)
    # the order of the sums does not change between calls
    assert torch.equal(gemm(ac, asc, wc, ws, TYPES[dtype]), y)


# enough tiles for those of 128 x 128 and of 256 x 256, with rows, columns and groups of k that end inside one
@pytest.mark.parametrize("m,n,k", [(513, 8328, 384), (1030, 10001, 640), (1537, 9000, 256)])
def test_gemm_large_tiles(m, n, k):
    test_gemm_exact(m, n, k)
    for dtype in TYPES:
        test_gemm(m, n, k, dtype)


@pytest.mark.parametrize("m", [1, 20, 64, 300])
def test_gemm_large_scales_and_nan(m):
    k, n = 512, 48
    ac, asc, wc, ws = operands(m, n, k, 9, 127, 128)
    asc[0, 3] = 255                     # row 0 is not a number
    ws[5, 2] = 255                      # nor is column 5
    asc[-1, :] = 127 + 60               # large and small factors that cancel
    ws[7, :] = 127 - 60
    a, w = plain.mx_values(ac, asc), plain.mx_values(wc, ws)
    got = gu.host(gemm(ac, asc, wc, ws))
    assert np.isnan(got[:, 5]).all() and (m == 1 or np.isnan(got[0]).all())
    want = a @ w.T
    fine = np.isfinite(want)
    assert np.array_equal(got[fine], want[fine].astype(np.float32))


@pytest.mark.parametrize("m", [3, 700])
def test_quantised_layer(m):
    """Quantise, multiply, as a layer is run; and the rotation on both sides leaves the product."""
    k, n = 1024, 640
    g = torch.Generator().manual_seed(3)
    x, wt = torch.randn(m, k, generator=g).bfloat16().to(gu.DEV), (0.05 * torch.randn(n, k, generator=g)).to(gu.DEV)
    for rotate in (False, True):
        w = tb.Mxfp4.quantise(wt, rotate)
        codes, scales = quant(x, rotate)
        y = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=gu.DEV)
        need = tb.tb_mxfp4_gemm_workspace_bytes(w, m)
        tb.tb_mxfp4_gemm(w, codes, scales, y, u8_out(need) if need else None)
        a = plain.mx_values(gu.host(codes), gu.host(scales))
        b = plain.mx_values(gu.host(w.codes), gu.host(w.scales))
        want, size = a @ b.T, np.abs(a) @ np.abs(b).T
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= 2 * k * U * size + 2.0 ** -8 * (1 + 1e-3) * np.abs(want))
        # the quantised product stands for the real one: relative error of two e2m1 roundings
        real = x.double().cpu().numpy() @ wt.double().cpu().numpy().T
        assert np.linalg.norm(want - real) < 0.25 * np.linalg.norm(real)


@pytest.mark.parametrize("m,n,k", [(1, 640, 1280), (48, 640, 1280), (300, 512, 2048)])
def test_layer_in_a_graph(m, n, k):
    g = torch.Generator(device=gu.DEV).manual_seed(4)
    x = torch.randn(m, k, generator=g, device=gu.DEV).bfloat16()
    w = tb.Mxfp4.quantise(torch.randn(n, k, generator=g, device=gu.DEV))
    codes, scales, y = u8_out(m, k // 2), u8_out(m, k // 32), gu.f32_out(m, n)
    need = tb.tb_mxfp4_gemm_workspace_bytes(w, m)
    ws = u8_out(need) if need else None

    def layer():
        tb.tb_mxfp4_quant(x, codes, scales)
        tb.tb_mxfp4_gemm(w, codes, scales, y, ws)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for r in range(3):
        x.copy_(torch.randn(m, k, generator=g, device=gu.DEV))
        layer()
        eager = y.clone()
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


def test_large_offsets():
    """Codes past 4 GiB: the last rows of a weight matrix of over 2^33 elements, against its own rows alone."""
    n, k = (1 << 20) + 1024, 8192
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB")
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=gu.DEV)
    scales = torch.randint(120, 124, (n, k // 32), dtype=torch.uint8, device=gu.DEV)
    for m in (1, 80):
        ac = torch.randint(0, 256, (m, k // 2), dtype=torch.uint8, device=gu.DEV)
        asc = torch.randint(120, 124, (m, k // 32), dtype=torch.uint8, device=gu.DEV)
        w, tail = tb.Mxfp4(codes, scales), tb.Mxfp4(codes[-1024:], scales[-1024:])
        y = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=gu.DEV)
        need = tb.tb_mxfp4_gemm_workspace_bytes(w, m)
        tb.tb_mxfp4_gemm(w, ac, asc, y, u8_out(need) if need else None)
        a = plain.mx_values(gu.host(ac), gu.host(asc))
        b = plain.mx_values(gu.host(tail.codes), gu.host(tail.scales))
        want, size = a @ b.T, np.abs(a) @ np.abs(b).T
        got = y[:, -1024:].double().cpu().numpy()
        assert np.all(np.abs(got - want) <= 2 * k * U * size + 2.0 ** -8 * (1 + 1e-3) * np.abs(want))


def test_binding_refusals():
    x = torch.randn(4, 256, device=gu.DEV)
    codes, scales, y = u8_out(4, 128), u8_out(4, 8), gu.f32_out(4, 32)
    w = tb.Mxfp4(u8_out(32, 128), u8_out(32, 8))

    def refuse(fn, *a, **kw):
        with pytest.raises(tb.TbError):
            fn(*a, **kw)
    refuse(tb.tb_mxfp4_quant, x.double(), codes, scales)
    refuse(tb.tb_mxfp4_quant, x.t(), codes, scales)
    refuse(tb.tb_mxfp4_quant, x, codes[:, :-1], scales)
    refuse(tb.tb_mxfp4_quant, x, codes, scales[:3])
    refuse(tb.tb_mxfp4_quant, x[:, :100].contiguous(), u8_out(4, 50), u8_out(4, 3))
    refuse(tb.tb_mxfp4_dequant, codes, scales, x.to(torch.int32))
    refuse(tb.Mxfp4, codes.view(torch.int8), scales)
    refuse(tb.Mxfp4, codes, scales[:, :4])
    refuse(tb.tb_mxfp4_gemm, w, codes, scales, y[:, :31].contiguous())
    refuse(tb.tb_mxfp4_gemm, w, codes[:3], scales, y)
    refuse(tb.tb_mxfp4_gemm, w, codes.cpu(), scales, y)
    refuse(tb.tb_mxfp4_gemm, w, codes, scales, y.double())
    assert (gu.host(codes) == 0xA5).all() and np.isnan(gu.host(y)).all()


def test_quantise_on_another_stream():
    """The new tensors belong to the stream that writes them: memory that the current stream has freed and
    may still be using is not handed to another."""
    n, k = 512, 4096
    x = torch.randn(n, k, device=gu.DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.empty(n, w, dtype=torch.uint8, device=gu.DEV) for w in (k // 2, k // 32)]
    places = {t.data_ptr() for t in freed}
    del freed
    for stream in (side, side.cuda_stream):
        w = tb.Mxfp4.quantise(x, stream=stream)
        assert w.codes.data_ptr() not in places and w.scales.data_ptr() not in places
        side.synchronize()
        want = tb.Mxfp4.quantise(x, stream=torch.cuda.current_stream().cuda_stream)
        assert torch.equal(w.codes, want.codes) and torch.equal(w.scales, want.scales)
        del w, want


# the row kernel with each number of rows, past 16 weight rows and past whole 256 elements of k, and the first
# that goes in tiles
@pytest.mark.parametrize("m,n,k", [(4, 100, 640), (5, 1000, 8064), (6, 33, 2432), (7, 250, 896), (8, 17, 384), (8, 9216, 5120), (8, 31, 8192),
                                   (8, 250, 896), (9, 250, 896), (8, 40, 8320)])
def test_gemm_few_rows(m, n, k):
    test_gemm_exact(m, n, k)
    for dtype in TYPES:
        test_gemm(m, n, k, dtype)
