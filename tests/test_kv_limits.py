"""Limits of the calls around the paged cache that need no GPU: no call here reaches a launch."""

import ctypes

import pytest

import ternary_weight_int8_tb_amd as tb
from tests.test_kv_abi import ATTN, L, attn_call, cache, heads  # noqa: F401 (L is a fixture)


def need(L, c, n, dtype, requests, tokens):
    return L.tb_attn_paged_workspace_bytes(ctypes.byref(c), n, dtype, requests, tokens)


def test_scale(L):
    """A scale whose product with log2 e fp32 does not hold is refused, not taken for infinity."""
    call = attn_call(L)
    for scale in (2.4e38, 2.6e38, 2.9e38, 3.3e38):
        assert call(scale=scale) == tb.TB_EINVAL, scale


def test_kernel_for_a_chunk_among_many_decodes(L):
    """250 decodes beside a chunk of 1000, at three heads a group: the rows of a request are few on average, and the chunk has many.
    The kernel for many rows runs, whose workspace is larger than that of the kernel for few."""
    call = attn_call(L)
    c = cache(kv=8, dim=128)
    few = need(L, c, 24, tb.TB_BF16, 1, 1)
    far = dict(zip(ATTN, [(i + 2) << 40 for i in range(5)]))
    q = heads(1 << 40, 3 * 24 * 128, 128, 24)
    assert need(L, c, 24, tb.TB_BF16, 251, 1250) > few
    assert call(q=q, c=cache(8 << 40, 9 << 40, kv=8, dim=128), requests=251, tokens=1250, ws_bytes=few, **far) == tb.TB_EINVAL


SIZES = [1, 2, 3, 4, 7, 8, 16, 17, 31, 32, 33, 40, 64, 100, 128, 129, 250, 256, 512, 1000, 1024, 2048, 4096]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,kv", [(16, 2), (24, 8), (8, 8), (32, 1), (128, 1), (1024, 1)])
def test_workspace_covers_smaller_calls(L, dim, n, kv):
    """A workspace for some requests and tokens is one for fewer of either."""
    c = cache(kv=kv, dim=dim)
    for dtype in (tb.TB_F32, tb.TB_BF16):
        sizes = [[need(L, c, n, dtype, r, t) for t in SIZES] for r in SIZES]
        for r in range(len(SIZES)):
            for t in range(len(SIZES)):
                assert 0 < sizes[r][t]
                assert r == 0 or sizes[r - 1][t] <= sizes[r][t], (SIZES[r], SIZES[t])
                assert t == 0 or sizes[r][t - 1] <= sizes[r][t], (SIZES[r], SIZES[t])


def test_workspace_is_enough(L):
    """What the call wants is never more than what the function says, and a workspace without room for any unit is refused."""
    c = cache(kv=2)
    for requests, tokens in ((1, 1), (3, 40), (250, 1249), (512, 512), (64, 128)):
        size = need(L, c, 16, tb.TB_BF16, requests, tokens)
        call = attn_call(L)
        far = dict(zip(ATTN, [(i + 2) << 40 for i in range(5)]))
        assert call(q=heads(1 << 40), c=cache(k=8 << 40, v=9 << 40), requests=requests, tokens=tokens, ws_bytes=4096, **far) == tb.TB_EINVAL
        assert size > 4096


def test_whole_numbers():
    """Arguments that 32 bits do not hold are refused; ctypes would cut them off (a window of 2^32 would be none)."""
    assert tb._int32("f", "n", 2 ** 31 - 1) == 2 ** 31 - 1 and tb._int32("f", "n", -2 ** 31) == -2 ** 31
    for v in (2 ** 31, 2 ** 32, 2 ** 32 + 16, -2 ** 31 - 1):
        with pytest.raises(tb.TbError) as e:
            tb._int32("f", "n", v)
        assert e.value.status == tb.TB_EINVAL
