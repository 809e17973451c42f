"""Keys whose scores are -inf for every row that sees them: weights of zero, and
rows that see no others give zeros.  Against the float64 oracle with those keys
left out (tolerances as in test_gpu_attn_prompt.py).
"""

import numpy as np
import pytest
import torch

import oracle.attention as ref
from test_gpu_attn_prompt import D, DEV, U, case, check, check_grads, eps, f64

pytestmark = pytest.mark.gpu


def without(q, k, v, gone, cu=None):
    """(o, lse, o_abs) with the keys of `gone` [B, T] taken out."""
    B, T, HQ, _ = q.shape
    G = HQ // k.shape[2]
    o, o_abs, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, HQ, T))
    for b in range(B):
        for lo, hi in ref.bounds_of(cu, T):
            seen = ref.causal(hi - lo) & ~gone[b, None, lo:hi]
            for h in range(HQ):
                kk = np.where(gone[b, lo:hi, None], 0.0, k[b, lo:hi, h // G])
                w, lse[b, h, lo:hi] = ref.head_weights(q[b, lo:hi, h], kk, D ** -0.5, seen)
                o[b, lo:hi, h], o_abs[b, lo:hi, h] = w @ v[b, lo:hi, h // G], w @ np.abs(v[b, lo:hi, h // G])
    return o, lse, o_abs


MASKED = [  # B, T, HQ, HKV, keys gone
    (1, 150, 4, 2, [(0, 64)]), (1, 300, 2, 1, [(0, 131)]), (2, 90, 2, 2, [(0, 90)]), (1, 200, 2, 1, [(0, 32), (70, 140)]),
    (1, 640, 2, 1, [(0, 640)]), (1, 900, 2, 1, [(0, 64)]), (1, 900, 2, 1, [(64, 128), (192, 256)]), (1, 900, 2, 1, [(0, 577)]),
]


@pytest.mark.parametrize("B,T,HQ,HKV,stretches", MASKED)
@pytest.mark.parametrize("kind", ["one -inf", "lowest"])
def test_scores_of_minus_infinity(gpu_lib, B, T, HQ, HKV, stretches, kind):
    q, k, v, up, _ = case(B, T, HQ, HKV, None, seed=400)
    q = q.abs() + 2.0 ** -6                        # every product with such a key is negative
    gone = np.zeros((B, T), bool)
    for lo, hi in stretches:
        gone[:, lo:hi] = True
        if kind == "lowest":
            k[:, lo:hi] = torch.finfo(torch.bfloat16).min     # the 128 products' sum overflows
        else:
            k[:, lo:hi, :, 5] = -float("inf")
    o, lse = gpu_lib.attn_prefill(q, k, v)
    want, wl, o_abs = without(f64(q), f64(k), f64(v), gone)
    ez = eps(f64(q), np.where(gone[..., None, None], 0.0, f64(k)), T)
    check(o, want, ((U + 2.1 * ez) * o_abs + U * np.abs(want)) * 1.01 + 1e-30, "o")
    seen = np.isfinite(wl)
    assert np.array_equal(np.isneginf(f64(lse)), ~seen)
    check(lse[torch.from_numpy(seen)], wl[seen], ez + 2.0 ** -22 * (1 + np.abs(wl[seen])), "lse")
    if kind == "one -inf":
        return                                     # a weight of zero times it is NaN in dQ
    # those keys, and rows that see no others, add nothing to any gradient
    grads = gpu_lib.attn_backward(q, k, v, o, lse, up, grad_dtype="float32")
    assert all(torch.isfinite(g).all() for g in grads)
    blind = torch.from_numpy(np.logical_and.accumulate(gone, 1))
    assert (grads[0][blind] == 0).all()
    assert all((g[torch.from_numpy(gone)] == 0).all() for g in grads[1:])
    if B == 1 and len(stretches) == 1 and stretches[0][1] < T:
        check_grads(grads, q, torch.where(torch.isfinite(k) & (k > -1e30), k, 0.0), v, up, [stretches[0][1], T], rounded=False)
