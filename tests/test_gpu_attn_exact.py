"""Attention over a paged cache where its contract can be told from a looser one: keys, queries and values are chosen so that
sums are exact or nearly so, and each bound is that of the contract alone."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import ternary_weight_int8_tb_amd as tb
from tests import gpu_util as gu
from tests.plain_kv import HALF_STEP, U
from tests.test_gpu_attn_paged import KINDS, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield


def said(c):
    torch.cuda.synchronize()
    return c.out[:c.tokens].double().cpu().numpy()


def fill(c, k, v):
    """k, v [requests][length][dim]: the keys and values of every head."""
    for s in range(len(c.lengths)):
        for j in range(c.lengths[s]):
            c.set(s, j, k=torch.as_tensor(k[s][j]), v=torch.as_tensor(v[s][j]))


@pytest.mark.parametrize("cache", ["f16", "bf16"])
@pytest.mark.parametrize("new", [5, 48])
def test_small_weights_of_fp32_rows(cache, new):
    """One key far above many equal ones, whose values alone are not zero: what a row returns is the sum of its smallest weights,
    and has their bits. d nats below the largest a weight keeps 22 bits, or an absolute error of 2^-38 of the largest (fp16)."""
    print(f"small weights {cache} new={new}", flush=True)
    n, heads, dim = 150, 8, 64
    c = Case([(n, new)], heads, 1, dim, 16, "f32", cache, seed=1)
    k, v = np.zeros((n, dim)), np.ones((n, dim))
    k[1:, 0] = -16.0
    v[0] = 0.0
    fill(c, [k], [v])
    # scores are products of two short numbers; d = 16 q, from 9.5 to 17
    d = 16 * (38 + np.arange(new * heads) % 31).reshape(new, heads) / 64.0
    c.q[:] = 0
    c.q[..., 0] = torch.from_numpy(d / 16).float()
    c.scale = 1.0
    c.upload().run()
    keys = n - new + np.arange(new)[:, None]           # beside the first
    t = np.exp(-d)
    want = keys * t / (1 + keys * t)
    # the parts 2^-22; the factor log2 e, its product with the scale and the score's with both: 3 U of d; the exponential 4 U; the
    # sums of `keys` alike, above and below, and of the waves and parts: U each; the division and the output: 8 U
    bound = want * (4 * U + 3 * U * d + 4 * U + 2 * (keys + 40) * U + 8 * U)
    if cache == "f16":
        bound = bound + want * 2.0 ** -38 / t
    off = np.abs(said(c) - want[..., None]) / bound[..., None]
    assert off.max() <= 1, off.max()


# Below these products of a maximum and the scale's factor, a row's scores are scaled and the maximum's product taken from them in
# one operation, so that all weights of one maximum have the rounding of that product: half a step of it
FUSED = {"bf16": 2.0 ** 13, "f16": 2.0 ** 10}


def base_error(score, kind):
    """The relative error between weights of two maxima near `score`"""
    at = score * np.log2(np.e)
    return 2 * at * 2.0 ** -24 * np.log(2) * 1.01 if at < FUSED[kind] else 0.0


SCORES = [700, 5600, 23170, 100003, 181071, 333337, 524287, 610101, 700001]


def keys_of(score, dim):
    """A key whose product with `query` is the whole number `score`, exactly, in either type: digits of at most 255"""
    k = np.zeros(dim)
    left, k[0] = score // 256, score % 256
    for i in range(1, 16):
        k[i] = min(left, 255)
        left -= int(k[i])
    assert left == 0
    return k


def query(dim):
    q = np.zeros(dim)
    q[0], q[1:16] = 1, 256
    return q


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_large_scores_of_two_maxima(kind, dim):
    """Scores that are whole numbers, and equal within each wave and each part: every weight is one, and what stands between
    the sums is exp of the maxima's difference, whatever their magnitude."""
    print(f"two maxima {kind} dim={dim}", flush=True)
    n = 640
    c = Case([(n, 1)] * len(SCORES), 2, 1, dim, 16, kind, kind, seed=2)
    group = np.arange(n) // 32 % 2          # blocks of 32 keys go to the waves in turn
    k = [np.where(group[:, None] == 1, keys_of(s + 1, dim), keys_of(s, dim)) for s in SCORES]
    v = np.repeat((1.0 - 2 * group)[:, None], dim, 1)
    fill(c, k, [v] * len(SCORES))
    c.q[:] = torch.from_numpy(query(dim))
    c.scale = 1.0
    got = said(c.upload().run())
    want = (1 - np.e) / (1 + np.e)
    # exp of the difference 1: 3 U and the exponential's 4 U, in each of two joins; sums of ones are exact; the division and the type
    bound = np.array([20 * U + base_error(s + 1, kind) for s in SCORES]) + HALF_STEP[kind] * abs(want)
    off = np.abs(got - want).max((1, 2)) / bound
    assert off.max() <= 1, off


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 40])
def test_large_scores_whose_maximum_moves(kind, dim, new):
    """Many equal scores, then a few that are 6 above them: the sums of the first are scaled by exp(-6)."""
    print(f"maximum moves {kind} dim={dim} new={new}", flush=True)
    n = 640
    c = Case([(n, new)] * len(SCORES), 4, 1, dim, 16, kind, kind, seed=3)
    top = (np.arange(n) >= 512) & (np.arange(n) % 32 == 0)
    rest = (np.arange(n) >= 512) & ~top
    k, v = [], np.repeat(np.where(top, -1.0, np.where(rest, 0.0, 1.0))[:, None], dim, 1)
    for s in SCORES:
        k.append(np.where(top[:, None], keys_of(s + 6, dim), np.where(rest[:, None], keys_of(s - 200, dim), keys_of(s, dim))))
    fill(c, k, [v] * len(SCORES))
    c.q[:] = torch.from_numpy(query(dim))
    c.scale = 1.0
    got = said(c.upload().run()).reshape(len(SCORES), new, -1)
    # one of the four lies among the last tokens' own keys
    high = np.array([top[:n - new + i + 1].sum() for i in range(new)]) * np.exp(6.0)
    want = (512 - high) / (512 + high)
    bound = (np.array([3 * 6 * U + 30 * U + base_error(s + 6, kind) for s in SCORES])[:, None] + HALF_STEP[kind] * np.abs(want))[..., None]
    off = np.abs(got - want[:, None]) / bound
    assert off.max() <= 1, off.max((1, 2))


@pytest.mark.parametrize("rows", ["f32", "bf16"])
@pytest.mark.parametrize("dim,new", [(64, 1), (128, 3), (256, 1), (256, 60)])
def test_large_values(rows, dim, new):
    """Values near the largest that bf16 holds: their mean is finite, and so is what is returned."""
    print(f"large values {rows} dim={dim} new={new}", flush=True)
    n = 700
    c = Case([(n, new)], 4, 2, dim, 16, rows, "bf16", seed=4)
    fill(c, [np.zeros((n, dim))], [np.full((n, dim), 1.5 * 2.0 ** 127)])
    got = said(c.upload().run())
    assert np.all(np.abs(got / (1.5 * 2.0 ** 127) - 1) <= (2 * n + 20) * U)
    # scores that grow, so that weights begin far above one
    c.k[:] = (torch.randn(c.k.shape, generator=torch.Generator().manual_seed(5)) * 2).to(c.k.dtype)
    c.upload().run()
    got = said(c)
    assert np.isfinite(got).all() and np.all(np.abs(got / (1.5 * 2.0 ** 127) - 1) <= (2 * n + 20) * U + (HALF_STEP["bf16"] if rows == "bf16" else 0))


@pytest.mark.parametrize("rows,cache", KINDS)
def test_tiny_and_large_scales(rows, cache):
    """Scales at both ends, with keys that are hidden: all weights alike, or one."""
    n, new, dim = 90, 20, 64
    for scale, unit in ((1e-44, 1.0), (2.0 ** -126, 1.0), (2.0 ** 126, 1.0), (1e-5, 2.0 ** -126), (2.0 ** -60, 2.0 ** -140), (2.0 ** 20, 2.0 ** 118),
                        (2.0 ** 120, 2.0 ** 60)):
        if unit != 1.0 and rows != "f32":
            continue
        print(f"scale {scale:g} of rows of {unit:g} {rows}/{cache}", flush=True)
        c = Case([(n, new)], 2, 1, dim, 16, rows, cache, seed=6)
        best = 37
        k = np.zeros((n, dim))
        k[:, 0] = -1.0 - np.arange(n) % 7
        k[best, 0] = 1.0
        v = np.arange(n)[:, None] % 5 + np.zeros((n, dim))
        fill(c, [k], [v])
        c.q[:] = 0
        c.q[..., 0] = unit
        c.scale = float(np.float32(scale))
        got = said(c.upload().run())
        alike = c.scale * unit < 1
        for i in range(new):
            seen = n - new + i + 1
            want = v[:seen, 0].mean() if alike else v[best, 0]
            # whole numbers: their sums are exact
            assert np.all(np.abs(got[i] - want) <= (HALF_STEP[rows] + 8 * U) * abs(want)), (scale, i, got[i, 0, 0], want)


@pytest.mark.parametrize("rows", ["f32", "bf16"])
@pytest.mark.parametrize("value", [2.0 ** -110, 2.0 ** -97, 1.5 * 2.0 ** 127])
@pytest.mark.parametrize("dim,new", [(64, 1), (128, 3), (256, 1), (256, 60)])
def test_values_of_any_magnitude(rows, value, dim, new):
    """Small bf16 values keep all their bits beside the room for large ones."""
    print(f"values of {value:g} {rows} dim={dim} new={new}", flush=True)
    n = 700
    c = Case([(n, new)], 4, 2, dim, 16, rows, "bf16", seed=7)
    x = (1 + np.arange(n) % 64 / 128)[:, None] + np.zeros((n, dim))
    if value > 1:
        x[:] = 1.0
    fill(c, [np.zeros((n, dim))], [x * value])
    got = said(c.upload().run())
    for i in range(new):
        want = x[:n - new + i + 1, 0].mean() * value
        # all weights are one: each product is exact, and so are the weights' sum and, up to 2^-149, that of the products
        assert np.all(np.abs(got[i] / want - 1) <= (n + 20) * U + HALF_STEP[rows] * 1.001), (got[i, 0, 0], want)
