"""What the norm bounds of latent_norms.py let pass and what they reject, on the CPU: gradients made with the kernels'
roundings pass, and each of a list of mistakes fails, at the shapes that the GPU tests use."""

import numpy as np
import pytest
import torch

import latent_norms
import oracle.latent as ref
from oracle.attention import head_weights

D, S, DQ = 128, 64, 192
SHAPES = [  # T, K, H, offsets of queries, of keys
    (32, 32, 2, None, None), (129, 129, 9, None, None), (517, 517, 3, None, None), (100, 333, 2, None, None),
    (700, 700, 1, None, None), (260, 900, 2, [0, 1, 100, 260], [0, 500, 600, 900]),
    (500, 560, 2, [3, 3, 170, 490], [5, 60, 200, 551]), (60, 120, 1, [40, 60, 20, 40], [80, 120, 30, 75]),
]


def inputs(T, K, H, seed=1):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*shape, generator=g).bfloat16().double().numpy()
            for shape in ((T, H, DQ), (K, H, D), (K, S), (K, H, D), (T, H, D))]


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().double().numpy()


def two_terms(x):
    return bf16(x) + bf16(x - bf16(x))


def gradients(x, cu, cu_kv, term=lambda y: y, rnd=lambda y: y, keep_delta=True, skip=None, rows=None):
    """The gradients with the kernels' roundings of operands (term) and results (rnd), or with a part left out."""
    q, k, s, v, up = x
    out = [np.zeros_like(y) for y in x[:4]]
    few = latent_norms._few_keys
    for lo, hi, klo, khi in ref.pairs(cu, cu_kv, len(q), len(k)):
        for h in range(q.shape[1]):
            qh, vh, uh, key = q[lo:hi, h], v[klo:khi, h], up[lo:hi, h], np.concatenate((k[klo:khi, h], s[klo:khi]), 1)
            w, _ = head_weights(qh, key, ref.SCALE, ref.seen(hi - lo, khi - klo))
            dw = uh @ vh.T
            delta = np.where(few(hi - lo, khi - klo), (w * dw).sum(1), (uh * rnd(rnd(w) @ vh)).sum(1))[:, None]
            ds = term(w * (dw - (delta if keep_delta else 0.0)))
            r = slice(None) if rows is None else rows
            out[0][lo:hi, h] = ref.SCALE * ds @ key
            dkey = ref.SCALE * ds[r].T @ qh[r]
            out[1][klo:khi, h] = dkey[:, :D]
            if h != skip:
                out[2][klo:khi] += dkey[:, D:]
            out[3][klo:khi, h] = term(w)[r].T @ uh[r]
    return [rnd(y) for y in out]


@pytest.mark.parametrize("T,K,H,cu,cu_kv", SHAPES)
def test_roundings_pass_and_mistakes_fail(T, K, H, cu, cu_kv):
    x = inputs(T, K, H)
    want = gradients(x, cu, cu_kv)
    full, _ = ref.latent_backward(*[a[None] for a in x], cu, cu_kv)
    for a, b in zip(want, full):
        inside = ~np.isnan(b[0])
        assert np.allclose(a[inside], b[0][inside], rtol=1e-9, atol=1e-12)
    args = dict(cu=cu, cu_kv=cu_kv)
    bound = latent_norms.bounds(*x, want, **args)
    worst = lambda got, b=bound: latent_norms.worst(got, want, b, **args)
    rounded = gradients(x, cu, cu_kv, bf16, bf16)
    assert 0.1 < worst(rounded) < 0.75

    # two terms, and the float32 results, are held to what they should be, which one term is not
    fine = latent_norms.bounds(*x, want, **args, rounded=False, u=2.0 ** -16)
    unrounded = gradients(x, cu, cu_kv, two_terms)
    assert worst(unrounded, fine) < 0.75
    if T <= 256 or K <= 256:
        coarse = gradients(x, cu, cu_kv, bf16)
        for i in range(4):
            assert worst([c if i == j else u for j, (c, u) in enumerate(zip(coarse, unrounded))], fine) > 1, i

    def fails(i, bad):
        got = list(rounded)
        got[i] = bad
        assert worst(got) > 1, i

    for i in range(4):
        fails(i, np.zeros_like(rounded[i]))
        fails(i, -rounded[i])
        fails(i, rounded[i] * 1.02)                            # a factor, a few roundings large
        nan = rounded[i].copy()
        nan[(cu if i == 0 else cu_kv or cu)[-1] - 1 if cu else 7] = np.nan
        fails(i, nan)
        fails(i, np.roll(rounded[i], 1, 0))                    # a row off
    one = rounded[0].copy()
    one[len(one) // 2:, 0] = 0                                 # half of one head
    fails(0, one)
    if T > 1:
        no_delta = gradients(x, cu, cu_kv, keep_delta=False)
        for i in range(3):
            fails(i, no_delta[i])
    fails(2, gradients(x, cu, cu_kv, bf16, bf16, skip=H - 1)[2])   # a head that did not enter the sum
    part = gradients(x, cu, cu_kv, rows=slice(0, T * 3 // 4)) if cu is None else None
    for i in (1, 2, 3):
        if part:
            fails(i, part[i])                                  # a part of the walk that did not


def test_one_head_of_many():
    """Of 70 heads one that did not enter the shared part's gradient."""
    x = inputs(450, 450, 70)
    want = gradients(x, None, None)
    bound = latent_norms.bounds(*x, want)
    rounded = gradients(x, None, None, bf16, bf16)
    assert latent_norms.worst(rounded, want, bound) < 0.75
    bad = rounded[:2] + [gradients(x, None, None, bf16, bf16, skip=33)[2]] + rounded[3:]
    assert latent_norms.worst(bad, want, bound) > 5
