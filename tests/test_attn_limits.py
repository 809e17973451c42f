"""Sizes past what one launch holds are refused before anything is enqueued (a
launch's threads are counted in 32 bits: 2^24 workgroups of 256 are too many).
Without a GPU; only refused calls are made."""

import pytest

import kda_gated_delta_amd as kda
from test_attn_abi import E_SHAPE, FAKE, backward, decode, prefill


@pytest.mark.parametrize("call", [prefill, backward])
def test_prompt_workgroups(call):
    for sizes in (dict(B=1 << 20, T=1, HQ=16, HKV=16), dict(B=1 << 18, T=129, HQ=32, HKV=8), dict(B=1 << 24, T=1, HQ=1, HKV=1),
                  dict(cu=FAKE, n=1 << 20, T=64, HQ=16, HKV=16), dict(cu=FAKE, n=2 ** 31 - 1, T=1, HQ=1, HKV=1)):
        assert call(qs=sizes["HQ"] * 128, ks=sizes["HKV"] * 128, vs=sizes["HKV"] * 128, **sizes) == E_SHAPE, sizes


def test_backward_counts_both_walks():
    # 2^19 sequences of a token: 16 heads' dQ and 16 heads' dK and dV
    assert backward(B=1 << 19, T=1, HQ=16, HKV=16, qs=2048, ks=2048, vs=2048) == E_SHAPE
    assert kda.attn_backward_workspace_size(1 << 19, 1, 16, 16) == 0
    assert kda.attn_backward_workspace_size((1 << 19) - 1, 1, 16, 16) == 8 * 16 * ((1 << 19) - 1)


def test_decode_workgroups():
    for N, HQ, HKV in ((1 << 20, 16, 16), (1 << 24, 1, 1), (1 << 21, 32, 8)):
        assert decode(N=N, HQ=HQ, HKV=HKV, qs=HQ * 128, stride=HKV * 64 * 128, wsb=1 << 50) == E_SHAPE
        assert kda.attn_decode_workspace_size(N, 1, HQ, HKV) == 0
    assert kda.attn_decode_workspace_size((1 << 20) - 1, 1, 16, 16) > 0
