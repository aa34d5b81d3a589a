"""Limits of the calls around the paged cache that need no GPU: no call here reaches a launch."""

import ctypes

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
