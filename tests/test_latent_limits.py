"""Sizes past what a launch of the kda_latent_* prompt entry points holds are refused before anything is enqueued: a
launch's threads are counted in 32 bits, so that 2^24 workgroups of 256 are too many, and 2^23 of the 512 that make
dK and dV.  Without a GPU; only refused calls are made."""

import pytest

import kda_gated_delta_amd as kda
from test_latent_abi import E_SHAPE, FAKE, backward

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
