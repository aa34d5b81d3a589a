"""Limits of the calls around the paged cache that need no GPU: no call here reaches a launch."""

import ternary_weight_int8_tb_amd as tb
from tests.test_kv_abi import L, attn_call  # noqa: F401 (L is a fixture)


def test_scale(L):
    """A scale whose product with log2 e fp32 does not hold is refused, not taken for infinity."""
    call = attn_call(L)
    for scale in (2.4e38, 2.6e38, 2.9e38, 3.3e38):
        assert call(scale=scale) == tb.TB_EINVAL, scale
