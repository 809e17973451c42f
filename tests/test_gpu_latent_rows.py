"""kda_latent_prefill, row by row: what lies behind a row does not change a bit of it.

A later token's key or shared part is replaced by a large one; the rows before it keep every bit of their outputs, and
all are right in float64.  Tolerances as in test_gpu_latent_prompt.py.
"""

import numpy as np
import pytest
import torch

import oracle.latent as ref
from test_gpu_attn_prompt import U, check, f64
from test_gpu_latent_prompt import case, eps

pytestmark = pytest.mark.gpu
SIZES = [  # T, K: one wave's rows, several tiles, keys before the queries, two sets of waves on a row tile
    (2, 2), (40, 40), (130, 130), (100, 171), (97, 700), (600, 600), (2100, 2117),
]


def places(T, K):
    """Tokens with rows before them: in the last tile, at its border, in others, the second row's."""
    return sorted({t for t in (K - 1, K - 2, K - 31, K - 33, K - 64, K - T // 2, K - T + 1) if t > K - T})


@pytest.mark.parametrize("T,K", SIZES)
def test_later_keys_that_are_large(gpu_lib, T, K):
    """A key along a later query: that row's maximum grows by far more than the rows before it notice."""
    q, k, s, v, _ = case(1, T, K, 2, seed=100)
    o, lse = gpu_lib.latent_prefill(q, k, s, v)
    for token in places(T, K):
        first = token - (K - T)                              # the first row that sees it
        for part in range(2):
            k2, s2 = k.clone(), s.clone()
            if part == 0:
                k2[0, token] = 2 * q[0, -1, :, :128]
            else:
                s2[0, token] = 4 * q[0, -1, 0, 128:]
            a, b = gpu_lib.latent_prefill(q, k2, s2, v)
            assert torch.equal(a[:, :first], o[:, :first]) and torch.equal(b[:, :, :first], lse[:, :, :first])
            x = [f64(t) for t in (q, k2, s2, v)]
            want, wl, o_abs = ref.latent_prefill(*x)
            ez = eps(*x[:3], ref.SCALE)
            check(a, want, ((U + 2.1 * ez) * o_abs + U * np.abs(want)) * 1.01, "o")
            check(b, wl, ez + 2.0 ** -22 * (1 + np.abs(wl)), "lse")
