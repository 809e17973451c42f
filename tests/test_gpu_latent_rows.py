"""kda_latent_prefill, row by row: what lies behind a row does not change a bit of it.

A later token's key, shared part and value are replaced by large ones, infinities and NaN; the rows before
it keep every bit of their outputs, and those from it on are right in float64, or not finite where the
definition is not.  Tolerances as in test_gpu_latent_prompt.py.
"""

import numpy as np
import pytest
import torch

import oracle.latent as ref
from test_gpu_attn_prompt import U, check, f64
from test_gpu_latent_prompt import case, eps, ints

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


@pytest.mark.parametrize("value", [2.0 ** 90, float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("T,K", SIZES)
def test_later_values(gpu_lib, T, K, value):
    """A value that is large or not finite, in some of its elements: the rows that do not see it, and what the others
    have in the other columns, are as they were."""
    q, k, s, v, _ = case(1, T, K, 2, seed=101)
    o, lse = gpu_lib.latent_prefill(q, k, s, v)
    columns = [0, 37, 70, 127]
    other = [d for d in range(128) if d not in columns]
    for token in places(T, K):
        first = token - (K - T)
        v2 = v.clone()
        v2[0, token, 1, columns] = value
        a, b = gpu_lib.latent_prefill(q, k, s, v2)
        assert torch.equal(b, lse) and torch.equal(a[:, :first], o[:, :first]) and torch.equal(a[:, :, 0], o[:, :, 0])
        assert torch.equal(a[..., other], o[..., other])
        if not np.isfinite(value):
            seen = a[0, first:, 1][:, columns].float()
            assert torch.isnan(seen).all() if np.isnan(value) else (seen == value).all()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("T,K", SIZES)
def test_later_keys_that_are_not_finite(gpu_lib, T, K, bad):
    q, k, s, v, _ = case(1, T, K, 2, seed=102)
    o, lse = gpu_lib.latent_prefill(q, k, s, v)
    for token in places(T, K):
        first = token - (K - T)
        for which in range(3):
            y = [t.clone() for t in (k, s, v)]
            y[which][0, token] = bad
            a, b = gpu_lib.latent_prefill(q, *y)
            assert torch.equal(a[:, :first], o[:, :first]) and torch.equal(b[:, :, :first], lse[:, :, :first])


def test_two_values_that_meet(gpu_lib):
    """Infinities of both signs: a row that sees both has NaN there, one that sees the first only has that."""
    T = K = 200
    q, k, s, v, _ = case(1, T, K, 2, seed=103)
    for first, second in ((3, 9), (5, 40), (130, 170), (70, 190)):
        v2 = v.clone()
        v2[0, first, 0, 5], v2[0, second, 0, 5] = float("inf"), -float("inf")
        a, _ = gpu_lib.latent_prefill(q, k, s, v2)
        got = a[0, :, 0, 5].float()
        assert torch.isfinite(got[:first]).all() and (got[first:second] == float("inf")).all()
        assert torch.isnan(got[second:]).all()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_packed(gpu_lib, value):
    """The same in sequences whose keys and rows are shifted against the tiles."""
    cu, cu_kv = [3, 70, 70, 171, 255], [10, 100, 130, 400, 484]
    c = dict(cu_seqlens=ints(cu), cu_seqlens_kv=ints(cu_kv))
    q, k, s, v, _ = case(1, 260, 490, 3, seed=104)
    o, lse = gpu_lib.latent_prefill(q, k, s, v, **c)
    inside = torch.zeros(260, dtype=torch.bool)
    inside[3:255] = True
    for lo, hi, klo, khi in ref.pairs(cu, cu_kv, 260, 490):
        for back in (1, 20, 50, 66):
            row, token = hi - back, khi - back
            if row <= lo:
                continue
            for which in range(3):
                y = [t.clone() for t in (k, s, v)]
                y[which][0, token] = value
                a, b = gpu_lib.latent_prefill(q, *y, **c)
                keep = inside.clone()
                keep[row:hi] = False
                assert torch.equal(a[:, keep], o[:, keep]) and torch.equal(b[:, :, keep], lse[:, :, keep])
