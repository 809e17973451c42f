"""Sizes whose workgroups do not fit the counts are refused by the kda_attn_* prompt entry points.  Without a GPU; only
refused calls are made."""

import pytest

import kda_gated_delta_amd as kda
from test_attn_abi import E_SHAPE, backward, prefill


@pytest.mark.parametrize("call", [prefill, backward])
def test_the_counts_do_not_overflow(call):
    """2^53 tiles times 2^11 heads are 0 in 64 bits, and 2^31 - 1 tokens a negative number of tiles in 32."""
    most = 2 ** 31 - 1
    for B, T, H in ((1 << 30, 1 << 30, 2048), (1, most, 65535), (2, most, 1)):
        assert call(B=B, T=T, HQ=H, HKV=H, qs=H * 128, ks=H * 128, vs=H * 128) == E_SHAPE
        assert kda.attn_backward_workspace_size(B, T, H, H) == 0
