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
