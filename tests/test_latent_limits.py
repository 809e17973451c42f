"""Sizes past what a launch of the kda_latent_* prompt entry points holds are refused before anything is enqueued: a
launch's threads are counted in 32 bits, so that 2^24 workgroups of 256 are too many, and 2^23 of the 512 that make
dK and dV.  Without a GPU; only refused calls are made."""

import pytest

import kda_gated_delta_amd as kda
from test_latent_abi import E_ALIGN, E_NULL, E_SHAPE, FAKE, NULL, OFF, backward, load, prefill, store

MOST = (1 << 23) - 1               # of 512 threads


@pytest.mark.parametrize("B,K,H", [(600000, 1, 16), (MOST + 1, 1, 1), (1 << 18, 129, 16)])
def test_workgroups_for_keys_alone(B, K, H):
    assert backward(B=B, T=0, K=K, H=H, qs=192 * H) == E_SHAPE
    assert kda.latent_backward_workspace_size(B, 0, K, H) == 0


def test_workgroups_for_packed_keys():
    assert backward(B=1, T=0, K=64, H=16, qs=192 * 16, cu=FAKE, cu_kv=FAKE, n=1 << 19) == E_SHAPE
    assert kda.latent_backward_workspace_size(1, 0, 64, 16, 1 << 19) == 0


def test_the_most_workgroups():
    assert kda.latent_backward_workspace_size(MOST, 0, 1, 1) == MOST * 64 * 4
    # queries and keys together, of one head
    assert kda.latent_backward_workspace_size(MOST, 1, 1, 1) > 0
    assert kda.latent_backward_workspace_size(MOST + 1, 1, 1, 1) == 0


def test_the_count_does_not_overflow():
    """2^53 tiles times 2^11 heads are 0 in 64 bits."""
    far = dict(B=1 << 30, H=2048, qs=2048 * 192)
    assert prefill(**far, T=1 << 30, K=1) == E_SHAPE
    for T, K in ((1 << 30, 1), (1, 1 << 30), (1 << 30, 1 << 30)):
        assert backward(**far, T=T, K=K) == E_SHAPE
        assert kda.latent_backward_workspace_size(1 << 30, T, K, 2048) == 0
    most = 2 ** 31 - 1
    assert prefill(B=2, T=most, K=1, H=4) == E_SHAPE and prefill(B=1, T=most, K=1, H=43690, qs=43690 * 192) == E_SHAPE
    for T, K in ((most, 1), (1, most)):
        assert backward(B=1, T=T, K=K, H=43690, qs=43690 * 192) == E_SHAPE


def test_the_most_heads():
    """A row of queries is 192 H elements of at most 2^23."""
    most = (1 << 23) // 192
    assert most == 43690
    for call in (prefill, backward):
        assert call(H=most, qs=192 * most, B=1 << 20) == E_SHAPE          # (for its workgroups)
        assert call(T=0, K=0, H=most, qs=192 * most) == 0
        for H in (most + 1, 65535):
            assert call(T=0, K=0, H=H, qs=1 << 23) == E_SHAPE and call(T=0, K=0, H=H, qs=192 * H) == E_SHAPE
    assert kda.latent_backward_workspace_size(1, 1, 1, most) > 0
    for H in (most + 1, 65535):
        assert kda.latent_backward_workspace_size(1, 1, 1, H) == 0


def test_the_most_tokens():
    """Of a store 8 to a workgroup, of a load 32: the last size that is taken fails for something else."""
    assert store(T=(1 << 27) - 8, slots=NULL) == E_NULL and store(T=(1 << 27) - 7, slots=NULL) == E_SHAPE
    assert load(T=(1 << 29) - 31) == E_SHAPE and load(T=(1 << 29) - 32, c=OFF) == E_ALIGN
