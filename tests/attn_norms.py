"""Bounds on the norm of an error in attention's gradients.

Elements' bounds add the roundings of all terms in magnitude and grow past the
gradients themselves on long walks.  Over thousands of elements the roundings,
independent of one another, add as squares.  With u = 2^-8 (half a bfloat16
step, relative) and every rounding's error taken at its largest, the error's norm
is at most u times the root of the sum of squares of
    what is rounded, times what it is multiplied with: dS with k (dQ) and q (dK),
    P with d_out (dV);
    what moves delta_i: o's own rounding and that of the weights behind it;
    the result's rounding, if it has one.
A rounding's root mean square is below half of its largest error, so that this
leaves a factor of two, by which no sum of independent errors exceeds its
expectation.
"""

import numpy as np

import oracle.attention as ref

U = 2.0 ** -8


def _norm2(x):
    return (x * x).sum(-1)


def gradient_terms(q, k, v, d_out, lo, hi, h, G, scale):
    """dS, P and the squares of delta's errors (over u) of one sequence and query head of [T, H, D] arrays."""
    qh, kh, vh, up = q[lo:hi, h], k[lo:hi, h // G], v[lo:hi, h // G], d_out[lo:hi, h]
    w, _ = ref.head_weights(qh, kh, scale, ref.causal(hi - lo))
    o, dw = w @ vh, up @ vh.T
    ds = w * (dw - (up * o).sum(1, keepdims=True))
    return ds, w, _norm2(up * o) + (w * w * dw * dw).sum(1), (qh, kh, vh, up)


def bounds(q, k, v, d_out, grads, cu=None, scale=None, rounded=True, u=U):
    """For dq, dk, dv [T, H, D] (float64, of one batch row): {(sequence's start, head): bound on the error's norm}."""
    T, HQ, D = q.shape
    HKV = k.shape[1]
    G = HQ // HKV
    scale = D ** -0.5 if scale is None else scale
    out = [{}, {}, {}]
    for lo, hi in ref.bounds_of(cu, T):
        if hi == lo:
            continue
        for g in range(HKV):
            dk2 = dv2 = 0.0
            for h in range(g * G, (g + 1) * G):
                ds, w, delta2, (qh, kh, _, up) = gradient_terms(q, k, v, d_out, lo, hi, h, G, scale)
                dq2 = scale ** 2 * (((ds * ds) @ _norm2(kh)).sum() + (delta2 * _norm2(w @ kh)).sum())
                out[0][lo, h] = dq2 + rounded * _norm2(grads[0][lo:hi, h]).sum()
                dk2 += scale ** 2 * (((ds * ds) + (w * w) * delta2[:, None]).sum(1) * _norm2(qh)).sum()
                dv2 += ((w * w).sum(1) * _norm2(up)).sum()
            out[1][lo, g] = dk2 + rounded * _norm2(grads[1][lo:hi, g]).sum()
            out[2][lo, g] = dv2 + rounded * _norm2(grads[2][lo:hi, g]).sum()
    return [{at: u * np.sqrt(x) for at, x in b.items()} for b in out]


def worst(got, want, bound, cu=None):
    """Largest error's norm over its bound, over tensors, sequences and heads; infinite where an error is not a number."""
    most = 0.0
    ends = dict((lo, hi) for lo, hi in ref.bounds_of(cu, want[0].shape[0]) if hi > lo)
    for g, w, b in zip(got, want, bound):
        for (lo, h), x in b.items():
            off = np.sqrt(_norm2((g - w)[lo:ends[lo], h]).sum())
            most = max(most, off / x if np.isfinite(off) else np.inf)
    return most
