"""What the norm bounds of attn_norms.py let pass and what they reject, on the
CPU: gradients made with the kernel's roundings pass, and each of a list of
mistakes fails, at the shapes that the GPU tests use."""

import numpy as np
import pytest
import torch

import attn_norms
import oracle.attention as ref

D = 128
SHAPES = [  # T, HQ, HKV, offsets
    (90, 4, 2, None), (517, 6, 2, None), (700, 4, 1, [0, 130, 700]), (1500, 8, 1, None),
]


def inputs(T, HQ, HKV, seed=1):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, h, D, generator=g).bfloat16().double().numpy() for h in (HQ, HKV, HKV, HQ)]


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().double().numpy()


def gradients(q, k, v, up, cu, rnd=lambda x: x, keep_delta=True, heads=None, rows=None):
    """The gradients with every rounding of the kernels (rnd), or with a part left out."""
    T, HQ, _ = q.shape
    G = HQ // k.shape[1]
    out = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    for lo, hi in ref.bounds_of(cu, T):
        for h in range(HQ):
            qh, kh, vh, do = q[lo:hi, h], k[lo:hi, h // G], v[lo:hi, h // G], up[lo:hi, h]
            w, _ = ref.head_weights(qh, kh, D ** -0.5, ref.causal(hi - lo))
            delta = (do * rnd(rnd(w) @ vh)).sum(1, keepdims=True)
            ds = rnd(w * (do @ vh.T - (delta if keep_delta else 0.0)))
            out[0][lo:hi, h] = D ** -0.5 * ds @ kh
            if heads is None or h in heads:
                r = slice(None) if rows is None else rows
                out[1][lo:hi, h // G] += D ** -0.5 * ds[r].T @ qh[r]
                out[2][lo:hi, h // G] += rnd(w)[r].T @ do[r]
    return [rnd(x) for x in out]


@pytest.mark.parametrize("T,HQ,HKV,cu", SHAPES)
def test_roundings_pass_and_mistakes_fail(T, HQ, HKV, cu):
    x = inputs(T, HQ, HKV)
    want = gradients(*x, cu)
    full, _ = ref.attn_backward(*[a[None] for a in x], cu)
    assert all(np.allclose(a, b[0], rtol=1e-9, atol=1e-12) for a, b in zip(want, full))
    bound = attn_norms.bounds(*x, want, cu)
    size = [min(b.values()) / np.linalg.norm(w) for b, w in zip(bound, want)]
    assert max(size) < 0.02, size
    rounded = gradients(*x, cu, rnd=bf16)
    assert 0.1 < attn_norms.worst(rounded, want, bound, cu) < 0.75

    def fails(i, bad):
        got = list(rounded)
        got[i] = bad
        assert attn_norms.worst(got, want, bound, cu) > 1, i

    for i in range(3):
        fails(i, np.zeros_like(rounded[i]))
        fails(i, -rounded[i])
        fails(i, rounded[i] * 1.02)                            # a factor, a few roundings large
        nan = rounded[i].copy()
        nan[T // 2, 0, 7] = np.nan
        fails(i, nan)
        one = rounded[i].copy()
        one[T // 2:, 0] = 0                                    # half of one head
        fails(i, one)
        fails(i, np.roll(rounded[i], 1, 0))                    # a row off
    no_delta = gradients(*x, cu, keep_delta=False)
    fails(0, no_delta[0])
    fails(1, no_delta[1])
    one_head = gradients(*x, cu, heads=range(1, HQ))           # a query head that did not enter the sum
    last_part = gradients(*x, cu, rows=slice(0, (T * 3) // 4)) if cu is None else None
    for i in (1, 2):
        fails(i, one_head[i])
        if last_part:
            fails(i, last_part[i])
